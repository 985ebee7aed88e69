// lrs_distill.hip -- distillation from a teacher's top logits (gfx950).
//
// With z = s / T, p = softmax(z) over a row of student logits s and q the
// teacher's mass on its top columns S (and q0 on all others, the tail, when its
// whole log-sum-exp is known), the row's loss is
//   sum_j q_j (log q_j - log p_j) + q0 (log q0 - log p0),
// and its gradient in z is A p_v - q_v on S and A p_v - q0 p_v / p0 elsewhere
// (A = all the teacher's mass: 1, or 0 in a row without any).  A row needs one
// pass for its sum of exponentials and, for the gradient, a second one.
//
// Sums over a row are in 32 bits for a thread's terms (at most 128, or one
// batch of loads where a row is longer) and in 64 bits from there on, as is
// everything there is once a row or a slot: the terms of a loss nearly cancel,
// and 1 - sum q loses a small tail in 32 bits.
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

constexpr int kDisBlock = 256;
constexpr double kLog2e = 1.44269504088896340736;
// Columns whose membership in S one workgroup holds as a bitmap at a time.
constexpr uint32_t kMapColumns = 65536;

// Of a piece of a row: its largest logit and the sum of exponentials relative to that.
struct Partial {
    double z;
    float m;
};

struct DisArgs {
    const void *logits;
    uint64_t stride;
    uint64_t rows;
    uint64_t first_row;   // of this launch
    uint32_t n, k;
    const void *tv;       // teacher's top logits
    uint64_t tv_stride;
    int tv_type;
    const void *ti;       // their columns
    uint64_t ti_stride;
    int ti_bytes;
    const float *tlse;    // the teacher's log-sum-exp by row, or null: no tail
    const float *weights; // by row, or null: 1 / rows
    double inv_t;
    float c, c_low;       // log2(e) / T, and what its rounding leaves
    uint32_t splits, split_len;
    Partial *partial;     // [rows][splits]: of the tail (of all, without one)
    float *stats;         // [rows][k + kStats]
    float *row_loss;
    float *loss;
    const float *loss_grad;
    void *grad;
    uint64_t grad_stride;
};

__device__ inline int64_t column_at(const DisArgs &a, uint64_t row, uint32_t j) {
    const uint64_t at = row * a.ti_stride + j;
    return a.ti_bytes == 8 ? static_cast<const int64_t *>(a.ti)[at] : static_cast<const int32_t *>(a.ti)[at];
}
__device__ inline float teacher_at(const DisArgs &a, uint64_t row, uint32_t j) {
    const uint64_t at = row * a.tv_stride + j;
    if (a.tv_type == kRowF32) return static_cast<const float *>(a.tv)[at];
    const uint16_t v = static_cast<const uint16_t *>(a.tv)[at];
    return a.tv_type == kRowBF16 ? Row<kRowBF16>::value(v) : Row<kRowF16>::value(v);
}
__device__ inline float weight_at(const DisArgs &a, uint64_t row) {
    return a.weights ? a.weights[row] : 1.0f / static_cast<float>(a.rows);
}

// x log2(e) / T less a reference, as an exponent of 2.  In 32-bit rows the
// rounding of the factor would show, by as much as |x| times its half step.
template <int T> __device__ inline float exponent(float x, float c, float c_low, float r) {
    const float e = fmaf(x, c, -r);
    return T == kRowF32 ? fmaf(x, c_low, e) : e;
}
// The factor that exponent() stands for.
template <int T> __device__ inline double factor_of(const DisArgs &a) {
    return T == kRowF32 ? static_cast<double>(a.c) + a.c_low : a.c;
}

// 2^d of a 64-bit d, to 32 bits.
__device__ inline double power_of_two(double d) {
    const double i = rint(d);
    return ldexp(static_cast<double>(__builtin_amdgcn_exp2f(static_cast<float>(d - i))),
                 static_cast<int>(fmax(fmin(i, 2000.0), -2000.0)));
}

// 2^d to about 44 bits: the series of exp on |y| <= ln 2 / 2, cut after
// y^11 / 11!.  Its coefficients go through scalar registers, made where they
// are used: in a loop that holds a row they would otherwise be kept in 22
// vector registers throughout.
__device__ inline double scalar(double v) {
    asm volatile("" : "+s"(v));
    return v;
}
constexpr double kLn2 = 0.693147180559945309417;
__device__ inline double exp2_64(double d) {
    d = d < -2000.0 ? -2000.0 : d;
    const double i = rint(d), y = (d - i) * scalar(kLn2);
    double p = scalar(1.0 / 39916800);
    p = fma(p, y, scalar(1.0 / 3628800));
    p = fma(p, y, scalar(1.0 / 362880));
    p = fma(p, y, scalar(1.0 / 40320));
    p = fma(p, y, scalar(1.0 / 5040));
    p = fma(p, y, scalar(1.0 / 720));
    p = fma(p, y, scalar(1.0 / 120));
    p = fma(p, y, scalar(1.0 / 24));
    p = fma(p, y, scalar(1.0 / 6));
    p = fma(p, y, 0.5);
    p = fma(p, y, 1.0);
    p = fma(p, y, 1.0);
    return ldexp(p, static_cast<int>(fmax(fmin(i, 2000.0), -2000.0)));
}
// z 2^d of a d of at most 0, exactly where d is whole.
__device__ inline double scaled(double z, double d) {
    if (d == rint(d)) return ldexp(z, static_cast<int>(fmax(d, -4000.0)));
    return z * exp2_64(d);
}
// log2 of a number in the range of 32 bits: the hardware's, and the rest from
// log(1 + e) = e - e^2 / 2 at e = v 2^-that - 1, below 2^-20.
__device__ inline double log2_64(double v) {
    const double y = __builtin_amdgcn_logf(static_cast<float>(v));
    const double e = v * exp2_64(-y) - 1.0;
    return y + fma(e * e, -0.5, e) * scalar(1.0 / kLn2);
}

// ---- rows over 256 KB ------------------------------------------------------
//
// A row's sum, its stats and its gradient are three launches: the row is read
// twice (1024 x 131072 fp32 step: 340 us, forward with a tail 112 us = 4.8 TB/s;
// 400 x 262144 bf16: 145 and 56 us = 3.7 TB/s, as an element takes the
// instructions of a 32-bit one at half the bytes).  The gradient is also the
// backward of every length: 515 x 32768 fp32 in 23 us = 5.8 TB/s, near the rate
// of a copy.

// One workgroup: the largest logit and the sum of exponentials of a piece of a row.
template <int T, bool TAIL>
__global__ __launch_bounds__(kDisBlock) void distill_sum_kernel(DisArgs a) {
    constexpr int kVec = Row<T>::kVec;
    __shared__ uint32_t map[TAIL ? kMapColumns / 32 : 1];
    __shared__ float wm[kDisBlock / kLanes];
    __shared__ double wz[kDisBlock / kLanes];
    const float c = a.c;
    using Stored = typename Row<T>::Stored;
    const auto power = [&](float below) { return __builtin_amdgcn_exp2f(exponent<T>(below, c, a.c_low, 0.f)); };
    for (uint64_t task = blockIdx.x; task < a.rows * a.splits; task += gridDim.x) {
        const uint64_t row = task / a.splits;
        const uint32_t first = static_cast<uint32_t>(task % a.splits) * a.split_len;
        const uint32_t last = min(a.n, first + a.split_len);
        const Stored *x = static_cast<const Stored *>(a.logits) + row * a.stride;
        float m = -INFINITY;
        double z = 0;
        if (weight_at(a, row) != 0.f) {
            for (uint32_t lo = first; lo < last; lo += kMapColumns) {
                const uint32_t hi = min(last, lo + kMapColumns);
                if (TAIL) {
                    __syncthreads();
                    for (uint32_t i = threadIdx.x; i < kMapColumns / 32; i += kDisBlock) map[i] = 0;
                    __syncthreads();
                    for (uint32_t j = threadIdx.x; j < a.k; j += kDisBlock) {
                        const int64_t col = column_at(a, row, j);
                        if (col >= lo && col < hi && teacher_at(a, row, j) > -INFINITY)
                            atomicOr(&map[(col - lo) / 32], 1u << ((col - lo) % 32));
                    }
                    __syncthreads();
                }
                const uint32_t vecs = (hi - lo) / kVec;
                const auto raise = [&](float top) {
                    if (top > m) {
                        if (m != -INFINITY) z *= power(m - top);
                        m = top;
                    }
                };
                // four loads at a time, one largest logit for all of them; their
                // sum alone is in 32 bits
                constexpr int kBatch = 4;
                for (uint32_t v = threadIdx.x; v < vecs; v += kBatch * kDisBlock) {
                    u32x4 w[kBatch];
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        const uint32_t at = min(v + u * kDisBlock, vecs - 1);
                        w[u] = load16(x + lo + static_cast<uint64_t>(at) * kVec);
                    }
                    float f[kBatch][kVec], top = m;
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        const uint32_t at = v + u * kDisBlock;
                        unpack16<T>(w[u], f[u]);
                        uint32_t out = at < vecs ? 0 : ~0u;  // elements that do not count
                        if (TAIL && at < vecs) out = map[at * kVec / 32] >> (at * kVec % 32);
#pragma unroll
                        for (int e = 0; e < kVec; ++e) {
                            if ((out >> e) & 1) f[u][e] = -INFINITY;
                            top = f[u][e] > top ? f[u][e] : top;
                        }
                    }
                    raise(top);
                    const float from = m == -INFINITY ? 0.f : m;
                    float part = 0;
#pragma unroll
                    for (int u = 0; u < kBatch; ++u)
#pragma unroll
                        for (int e = 0; e < kVec; ++e) part += power(f[u][e] - from);
                    z += part;
                }
                const uint32_t t = vecs * kVec + threadIdx.x;
                if (t < hi - lo && (!TAIL || !((map[t / 32] >> (t % 32)) & 1))) {
                    const float f = Row<T>::value(x[lo + t]);
                    raise(f);
                    if (f != -INFINITY) z += power(f - m);
                }
            }
        }
        // the threads' sums, relative to the largest logit of all
        float top = wave_max(m);
        __syncthreads();
        if (threadIdx.x % kLanes == 0) wm[threadIdx.x / kLanes] = top;
        __syncthreads();
        for (int w = 0; w < kDisBlock / kLanes; ++w) top = fmaxf(top, wm[w]);
        if (m != -INFINITY) z *= exp2_64((static_cast<double>(m) - top) * factor_of<T>(a));
        z = wave_sum(z);
        if (threadIdx.x % kLanes == 0) wz[threadIdx.x / kLanes] = z;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kDisBlock / kLanes; ++w) z += wz[w];
            a.partial[task] = Partial{z, top};
        }
    }
}

// A product rounded by itself, not within a fused difference: where logits are
// huge, equal ones have to cancel.
__device__ inline double times(double a, double b) {
    double p = a * b;
    asm("" : "+v"(p));
    return p;
}

// A reference of up to 2^20 is a whole number: m c in 32 bits is within 2^-4 of
// m times the factor there, so exponents of the largest logits stay near 0.
// Beyond, the rounding of m c grows with it (at 2^32 to 2^7, and 2^127 is past
// what 32 bits hold), so exponents are (x - m) c, whose difference is exact for
// all that have a share, and the reference is m times the factor in 64 bits.
// The half keeps whole references, after their rounding, from passing 2^20.
constexpr double kWholeReference = 0x1p20;
__device__ inline bool huge_logit(float m, float c) {
    return fabsf(m) < INFINITY && !(fabsf(m * c) < static_cast<float>(kWholeReference) + 0.5f);
}
// The logit that exponents with this reference are relative to, 0 where they are relative to the reference itself.
__device__ inline float base_of(double reference, double factor) {
    const bool huge = fabs(reference) < INFINITY && fabs(reference) > kWholeReference;
    return huge ? static_cast<float>(reference / factor) : 0.f;
}

// What a row's gradient needs: off S it is f 2^((x - b) c - r) with b, r and f
// the first three stats (r whole and b 0, or b the largest logit and r 0 where
// that is huge), at slot j's column stats[3 + j], all before weight / T.
constexpr uint32_t kStats = 3;
__device__ inline void write_stats(float *stats, double reference, float base, double f) {
    stats[0] = base;
    stats[1] = base != 0.f ? 0.f : static_cast<float>(reference);
    stats[2] = static_cast<float>(f);
}

// One wave a row: the teacher's masses, the loss and the stats.
template <int T>
__global__ __launch_bounds__(kLanes) void distill_row_kernel(DisArgs a) {
    __shared__ double q[LRS_MAX_TOPK];
    __shared__ int32_t col[LRS_MAX_TOPK];
    using Stored = typename Row<T>::Stored;
    const int lane = threadIdx.x;
    const double inv_t = a.inv_t;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float *stats = a.stats + row * (a.k + kStats);
        if (weight_at(a, row) == 0.f) {
            for (uint32_t j = lane; j < a.k + kStats; j += kLanes) stats[j] = 0.f;
            if (lane == 0 && a.row_loss) a.row_loss[row] = 0.f;
            continue;
        }
        const Stored *x = static_cast<const Stored *>(a.logits) + row * a.stride;
        const bool tail = a.tlse != nullptr;
        // the row's sums
        float m = -INFINITY;
        for (uint32_t s = lane; s < a.splits; s += kLanes) m = fmaxf(m, a.partial[row * a.splits + s].m);
        m = wave_max(m);
        double z = 0;
        for (uint32_t s = lane; s < a.splits; s += kLanes) {
            const Partial p = a.partial[row * a.splits + s];
            z += p.m == -INFINITY ? p.z : p.z * exp((static_cast<double>(p.m) - m) * inv_t);
        }
        z = wave_sum(z);
        // the counted slots
        __syncthreads();
        float tm = -INFINITY;
        for (uint32_t j = lane; j < a.k; j += kLanes) {
            const int64_t at = column_at(a, row, j);
            const float t = teacher_at(a, row, j);
            const bool counts = at >= 0 && at < a.n && t > -INFINITY;
            col[j] = counts ? static_cast<int32_t>(at) : -1;
            if (counts) tm = fmaxf(tm, t);
        }
        tm = wave_max(tm);
        __syncthreads();
        const double ref = tail ? a.tlse[row] : tm * inv_t;
        double sum = 0;
        uint32_t distinct = 0;
        float sm = -INFINITY;  // the largest student logit on S
        for (uint32_t j = lane; j < a.k; j += kLanes) {
            const bool counts = col[j] >= 0;
            const double e = counts ? exp(teacher_at(a, row, j) * inv_t - ref) : 0;
            q[j] = e;
            sum += e;
            bool again = false;
            for (uint32_t i = 0; i < j; ++i) again |= col[i] == col[j];
            distinct += counts && !again;
            if (counts) sm = fmaxf(sm, Row<T>::value(x[col[j]]));
        }
        sum = wave_sum(sum);
        distinct = wave_sum(distinct);
        sm = wave_max(sm);
        double scale = 1, q0 = 0, mass = sum;
        if (tail) {
            q0 = fmax(0.0, 1.0 - sum);
            if (distinct == a.n || (m == -INFINITY && q0 <= 0x1p-20)) q0 = 0;
        } else {
            scale = sum > 0 ? 1 / sum : 0;
            mass = sum > 0 ? 1 : 0;
        }
        // log-sum-exp of the whole row: the tail's and S's (without a tail z covers the row)
        float top = m;
        double whole = z;
        if (tail) {
            top = fmaxf(m, sm);
            double on = 0;
            for (uint32_t j = lane; j < a.k; j += kLanes) {
                bool again = false;
                for (uint32_t i = 0; i < j; ++i) again |= col[i] == col[j];
                if (col[j] < 0 || again) continue;
                const float s = Row<T>::value(x[col[j]]);
                if (s != -INFINITY) on += exp((static_cast<double>(s) - top) * inv_t);
            }
            whole = wave_sum(on) + (m == -INFINITY ? z : z * exp((static_cast<double>(m) - top) * inv_t));
        }
        // relative to `top`, which may be huge
        const double lse = top == -INFINITY ? -INFINITY : log(whole);
        const double lse0 = m == -INFINITY ? -INFINITY : (static_cast<double>(m) - top) * inv_t + log(z);
        const double a_mass = mass + q0;
        double loss = 0;
        __syncthreads();
        for (uint32_t j = lane; j < a.k; j += kLanes) {
            float g = 0;
            if (col[j] >= 0) {
                const double s = Row<T>::value(x[col[j]]);
                const double qj = q[j] * scale;
                if (qj > 0) loss += s == -INFINITY ? INFINITY : qj * (log(qj) - ((s - top) * inv_t - lse));
                double all = 0;  // what the teacher puts on this column, if it is there more than once
                for (uint32_t i = 0; i < a.k; ++i)
                    if (col[i] == col[j]) all += q[i] * scale;
                const double p = s == -INFINITY ? 0 : exp((s - top) * inv_t - lse);
                g = static_cast<float>(a_mass * p - all);
            }
            stats[kStats + j] = g;
        }
        loss = wave_sum(loss);
        if (lane == 0) {
            if (q0 > 0) loss += m == -INFINITY ? INFINITY : q0 * (log(q0) - (lse0 - lse));
            if (a.row_loss) a.row_loss[row] = static_cast<float>(loss);
            // 2^((x - b) c - r) in place of exp((x - m) / T)
            const float c = a.c;
            const double exact = times(m, factor_of<T>(a));
            const double r = m == -INFINITY ? 0 : huge_logit(m, c) ? exact : rintf(m * c);
            double f = 0;
            if (m != -INFINITY) {
                f = a_mass * exp((static_cast<double>(m) - top) * inv_t - lse);
                if (q0 > 0) f -= q0 / z;
                f *= exp2(r - exact);
            }
            write_stats(stats, r, base_of(r, factor_of<T>(a)), f);
        }
    }
}

// The weighted sum of the row losses, in a fixed order.
__global__ __launch_bounds__(1024) void distill_loss_kernel(DisArgs a) {
    __shared__ double part[1024 / kLanes];
    double s = 0;
    for (uint64_t r = threadIdx.x; r < a.rows; r += 1024) {
        const float w = weight_at(a, r);
        if (w != 0.f) s += static_cast<double>(w) * a.row_loss[r];
    }
    s = wave_sum(s);
    if (threadIdx.x % kLanes == 0) part[threadIdx.x / kLanes] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0;
        for (int w = 0; w < 1024 / kLanes; ++w) s += part[w];
        *a.loss = static_cast<float>(s);
    }
}

// One workgroup: the gradient of a piece of a row.
template <int T>
__global__ __launch_bounds__(kDisBlock) void distill_grad_kernel(DisArgs a) {
    constexpr int kVec = Row<T>::kVec;
    using Stored = typename Row<T>::Stored;
    const float c = a.c;
    const float up = a.loss_grad ? *a.loss_grad : 1.f;
    for (uint64_t task = blockIdx.x; task < a.rows * a.splits; task += gridDim.x) {
        const uint64_t row = task / a.splits;
        const uint32_t first = static_cast<uint32_t>(task % a.splits) * a.split_len;
        const uint32_t len = min(a.n - first, a.split_len);
        const Stored *x = static_cast<const Stored *>(a.logits) + row * a.stride + first;
        Stored *g = static_cast<Stored *>(a.grad) + row * a.grad_stride + first;
        const float *stats = a.stats + row * (a.k + kStats);
        const float w = weight_at(a, row);
        const uint32_t vecs = len / kVec;
        if (w == 0.f) {  // whatever its logits hold
            for (uint32_t v = threadIdx.x; v < vecs; v += kDisBlock) store16(g + static_cast<uint64_t>(v) * kVec, u32x4{0, 0, 0, 0});
            const uint32_t t = vecs * kVec + threadIdx.x;
            if (t < len) g[t] = 0;
            continue;
        }
        const float b = stats[0], r = stats[1], scale = up * w * static_cast<float>(a.inv_t), f = stats[2] * scale;
        for (uint32_t v = threadIdx.x; v < vecs; v += kDisBlock) {
            float e[kVec];
            unpack16<T>(load16(x + static_cast<uint64_t>(v) * kVec), e);
            for (int i = 0; i < kVec; ++i) e[i] = __builtin_amdgcn_exp2f(exponent<T>(e[i] - b, c, a.c_low, r)) * f;
            store16(g + static_cast<uint64_t>(v) * kVec, pack16<T>(e));
        }
        const uint32_t t = vecs * kVec + threadIdx.x;
        if (t < len) g[t] = Row<T>::pattern(__builtin_amdgcn_exp2f(exponent<T>(Row<T>::value(x[t]) - b, c, a.c_low, r)) * f);
        // the teacher's columns over what was written there
        __syncthreads();
        for (uint32_t j = threadIdx.x; j < a.k; j += kDisBlock) {
            const int64_t at = column_at(a, row, j) - first;
            if (at >= 0 && at < len && teacher_at(a, row, j) > -INFINITY) g[at] = Row<T>::pattern(stats[kStats + j] * scale);
        }
        __syncthreads();
    }
}

// ---- a whole row in one workgroup's registers ------------------------------

// LDS of a held row: what is known of the k slots, the partial sums and the
// bitmap of the columns in S (last).
struct HeldLds {
    static constexpr uint32_t kFixed = 512;
    __host__ __device__ static uint32_t slots(uint32_t k) { return (k + 1) / 2 * 2; }
    __host__ __device__ static uint32_t map(uint32_t k) { return kFixed + slots(k) * 20; }
    __host__ __device__ static uint32_t bytes(uint32_t k, uint32_t n) { return map(k) + (n + 31) / 32 * 4; }
};

// One workgroup of B threads a row, V loads of 16 bytes a thread.  With a
// gradient the row stays in registers from its one read to its one write, both
// past the caches' usual order (nontemporal): nothing of it is read again.
// Without, four loads are on their way at a time and twice the rows are on a CU.
// Exponents are in units of log 2 with c = log2(e) / T, in 16-bit rows rounded
// to 32 bits, everywhere the same c, and references to them are whole numbers R: the sums of
// 2^(x c - R) of two waves join exactly, and log2 sum 2^(x c) = R + log2(sum).
//
// Bound by HBM where rows are long and many: 4096 x 131072 bf16 step 421 us = 5.1
// TB/s, where a copy of the rows in the same form takes 367 us; the rest is the
// chain from the last load to the first store (joins, the teacher's terms in 64
// bits by one wave, the factor), which a second row on the CU would hide and two
// rows of 256 KB do not fit.  1031 x 50021 fp16 step with a tail 50 us, forward
// 1024 x 65536 fp16 with a tail 27 us = 4.9 TB/s (32 us when it stayed in
// registers).  Keeping only the first loads with a gradient, too, and reading
// the rest again costs 0 to 18%.
template <int T, int B, int V, bool GRAD>
__global__ __launch_bounds__(B, GRAD ? 4 : 8) void distill_held_kernel(DisArgs a) {
    constexpr int kVec = Row<T>::kVec;
    constexpr int kWaves = B / kLanes;
    using Stored = typename Row<T>::Stored;
    extern __shared__ __align__(16) uint8_t lds[];
    double *wz = reinterpret_cast<double *>(lds);                  // by wave
    double *wr = reinterpret_cast<double *>(lds + 128);
    double *out = reinterpret_cast<double *>(lds + 256);           // the row's reference, the factor
    double *teacher = reinterpret_cast<double *>(lds + 272);       // its reference, its mass on S
    uint32_t *again = reinterpret_cast<uint32_t *>(lds + 288);     // a column is there more than once
    uint32_t *columns = again + 1;                                 // distinct ones
    float *base = reinterpret_cast<float *>(columns + 1);          // the logit that the row's exponents are relative to
    const uint32_t slots = HeldLds::slots(a.k);
    double *q = reinterpret_cast<double *>(lds + HeldLds::kFixed);
    int32_t *col = reinterpret_cast<int32_t *>(q + slots);
    float *sl = reinterpret_cast<float *>(col + slots);            // the student's logit, then the slot's gradient
    float *tl = sl + slots;
    uint32_t *map = reinterpret_cast<uint32_t *>(lds + HeldLds::map(a.k));
    const uint32_t tid = threadIdx.x, vecs = a.n / kVec;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kLanes);
    const uint32_t n = a.n, k = a.k, rest = vecs * kVec + tid;
    const float c = a.c;
    const bool tail = a.tlse != nullptr;
    const uint32_t none = T == kRowF16 ? 0xFC00FC00u : T == kRowBF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf

    const int lane = tid % kLanes;
    const uint64_t row = a.first_row + xcd_chunk(blockIdx.x, gridDim.x);
    const Stored *x = static_cast<const Stored *>(a.logits) + row * a.stride;
    Stored *g = static_cast<Stored *>(a.grad) + row * a.grad_stride;
    float *stats = a.stats ? a.stats + row * (k + kStats) : nullptr;
    const float weight = weight_at(a, row);
    if (weight == 0.f) {  // whatever its logits hold
        if (stats)
            for (uint32_t j = tid; j < k + kStats; j += B) stats[j] = 0.f;
        if (tid == 0) a.row_loss[row] = 0.f;
        if (GRAD) {
            for (uint32_t v = tid; v < vecs; v += B) store16_once(g + static_cast<uint64_t>(v) * kVec, u32x4{0, 0, 0, 0});
            if (rest < n) g[rest] = 0;
        }
        return;
    }
    // the first slot of every thread, then the row: a scalar base, one offset for all
    int64_t at = tid < k ? column_at(a, row, tid) : -1;
    float t = tid < k ? teacher_at(a, row, tid) : 0.f;
    const auto below = [&](uint32_t count, int u) { return static_cast<int>(tid) < static_cast<int>(count) - u * B; };
    const auto load = [&](int u) {
        const uint8_t *p = reinterpret_cast<const uint8_t *>(x + u * B * kVec) + tid * 16;
        u32x4 w{none, none, none, none};
        if (below(vecs, u)) w = load16_once(p);
        return w;
    };
    // with a gradient the whole row stays; else its first loads do, and others
    // are read as they are used
    constexpr int kKeep = GRAD || V <= 4 ? V : 4;
    u32x4 v[kKeep];
#pragma unroll
    for (int u = 0; u < kKeep; ++u) v[u] = load(u);
    float over = rest < n ? Row<T>::value(x[rest]) : -INFINITY;
    float r = 0.f, factor = 1.f, m = 0.f;
    uint32_t sign = 0;
    bool huge = false;
    double reference = 0;
    for (uint32_t i = tid; i < (n + 31) / 32; i += B) map[i] = 0;
    if (tid == 0) *again = 0;
    __syncthreads();
    Stored raw = 0;
#pragma unroll 1
    for (uint32_t j = tid; j < k; j += B) {
        if (j != tid) {
            at = column_at(a, row, j);
            t = teacher_at(a, row, j);
        }
        const bool counts = at >= 0 && at < n && t > -INFINITY;
        col[j] = counts ? static_cast<int32_t>(at) : -1;
        tl[j] = t;
        if (counts) {
            const uint32_t bit = 1u << (at % 32);
            if (atomicOr(&map[at / 32], bit) & bit) *again = 1;
            if (j == tid) raw = x[at];
        }
    }
    __syncthreads();
    // the teacher's masses, while the row is on its way
    if (wave == 0) {
        double sum = 0;
        uint32_t distinct = 0;
        float tm = -INFINITY;
#pragma unroll 1
        for (uint32_t j = lane; j < k; j += kLanes)
            if (col[j] >= 0) tm = fmaxf(tm, tl[j]);
        tm = wave_max(tm);
        const double known = tail ? a.tlse[row] : tm == -INFINITY ? 0.0 : static_cast<double>(tm) * a.inv_t;
#pragma unroll 1
        for (uint32_t j = lane; j < k; j += kLanes) {
            const double e = col[j] >= 0 ? exp2_64((static_cast<double>(tl[j]) * a.inv_t - known) * scalar(1.0 / kLn2)) : 0;
            q[j] = e;
            sum += e;
            bool first = col[j] >= 0;
            if (*again)
#pragma unroll 1
                for (uint32_t i = 0; i < j; ++i) first &= col[i] != col[j];
            distinct += first;
        }
        sum = wave_sum(sum);
        distinct = wave_sum(distinct);
        if (lane == 0) {
            teacher[0] = known;
            teacher[1] = sum;
            *columns = distinct;
        }
    }
    // S does not count in the sum of a tail
    const auto without_s = [&](u32x4 &w, int u) {
        if (below(vecs, u)) {
            const uint32_t bits = (map[u * (B * kVec / 32) + tid * kVec / 32] >> (tid * kVec % 32)) & ((1u << kVec) - 1);
            if (bits) {
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if ((bits >> e) & 1) {
                        if (T == kRowF32) w[e % 4] = none;
                        else w[e / 2] = e & 1 ? (w[e / 2] & 0xFFFFu) | (none & 0xFFFF0000u)
                                              : (w[e / 2] & 0xFFFF0000u) | (none & 0xFFFFu);
                    }
            }
        }
    };
    if (tail) {
#pragma unroll
        for (int u = 0; u < kKeep; ++u) without_s(v[u], u);
        if (rest < n && ((map[rest / 32] >> (rest % 32)) & 1)) over = -INFINITY;
    }
    // each pass unpacks the held words anew: their floats would take twice the registers
    const auto anew = [&]() {
#pragma unroll
        for (int u = 0; u < kKeep; ++u) asm volatile("" : "+v"(v[u]));
    };
    const auto larger = [&](float m, u32x4 w) {
        float f[kVec];
        unpack16<T>(w, f);
#pragma unroll
        for (int e = 0; e < kVec; ++e) m = f[e] > m ? f[e] : m;
        return m;
    };
    // f for every load of the row, four on their way at a time where it does not stay
    const auto each = [&](auto f) {
#pragma unroll
        for (int u = 0; u < kKeep; ++u) f(v[u]);
        if constexpr (kKeep < V) {
#pragma unroll 1
            for (int b = kKeep; b < V; b += kKeep) {
                u32x4 t[kKeep];
#pragma unroll
                for (int u = 0; u < kKeep; ++u) t[u] = load(b + u);
#pragma unroll
                for (int u = 0; u < kKeep; ++u) {
                    if (tail) without_s(t[u], b + u);
                    f(t[u]);
                }
            }
        }
    };
    const auto sum_of = [&](auto term) {
        float part = term(over);
        each([&](u32x4 w) {
            float f[kVec];
            unpack16<T>(w, f);
#pragma unroll
            for (int e = 0; e < kVec; ++e) part += term(f[e]);
        });
        return wave_sum(static_cast<double>(part));
    };
    const auto power = [&](float x) { return __builtin_amdgcn_exp2f(exponent<T>(x, c, a.c_low, r)); };
    // A sum needs a reference near its largest term, not at it: first one from
    // the first load of each lane, and if the sum then leaves its range, the
    // largest of all.
    m = wave_max(larger(over, v[0]));
    r = m == -INFINITY || huge_logit(m, c) ? 0.f : rintf(m * c);
    anew();
    double z_wave = sum_of(power);
    anew();
    reference = r;
    if (!(z_wave >= 0x1p-20 && z_wave <= 0x1p40)) {
        m = over;
        each([&](u32x4 w) { m = larger(m, w); });
        m = wave_max(m);
        huge = huge_logit(m, c);
        r = m == -INFINITY || huge ? 0.f : rintf(m * c);
        reference = m == -INFINITY ? -INFINITY : huge ? times(m, factor_of<T>(a)) : r;
    }
    anew();
    if (huge) z_wave = sum_of([&](float x) { return __builtin_amdgcn_exp2f(exponent<T>(x - m, c, a.c_low, 0.f)); });
    else if (!(z_wave >= 0x1p-20 && z_wave <= 0x1p40)) z_wave = sum_of(power);
    anew();
    if (lane == 0) {
        wz[wave] = z_wave;
        wr[wave] = reference;
    }
#pragma unroll 1
    for (uint32_t j = tid; j < k; j += B)
        sl[j] = col[j] < 0 ? -INFINITY : Row<T>::value(j == tid ? raw : x[col[j]]);
    __syncthreads();
    if (wave == 0) {
        const double cd = factor_of<T>(a);
        // the row's sum (off S where there is a tail)
        double R = lane < kWaves ? wr[lane] : -INFINITY;
        double z = lane < kWaves ? wz[lane] : 0;
        const double mine = R, known = teacher[0], sum = teacher[1];
        R = wave_max(R);
        const bool empty = R == -INFINITY;
        if (mine != -INFINITY) z = scaled(z, mine - R);
        z = wave_sum(z);
        double scale = 1, q0 = 0, mass = sum;
        if (tail) {
            q0 = fmax(0.0, 1.0 - sum);
            if (*columns == n || (empty && q0 <= 0x1p-20)) q0 = 0;
        } else {
            scale = sum > 0 ? 1 / sum : 0;
            mass = sum > 0 ? 1 : 0;
        }
        // the whole row's
        double whole_r = empty ? 0.0 : R;
        double whole = z;
        if (tail) {
            float sm = -INFINITY;
#pragma unroll 1
            for (uint32_t j = lane; j < k; j += kLanes) sm = fmaxf(sm, sl[j]);
            sm = wave_max(sm);
            if (sm != -INFINITY) whole_r = fmax(empty ? -INFINITY : R, rint(times(sm, cd)));
            double on = 0;
#pragma unroll 1
            for (uint32_t j = lane; j < k; j += kLanes) {
                bool first = col[j] >= 0 && sl[j] != -INFINITY;
                if (first && *again)
#pragma unroll 1
                    for (uint32_t i = 0; i < j; ++i) first &= col[i] != col[j];
                if (first) on += power_of_two(times(sl[j], cd) - whole_r);
            }
            on = wave_sum(on);
            whole = on + (empty ? z : scaled(z, R - whole_r));
        }
        // the logarithms, a lane each
        const double of = lane == 0 ? whole : lane == 1 ? z : lane == 2 ? q0 : sum;
        const double logs = log2_64(of);
        // log-sum-exps stay apart from their references, which may be huge
        const double lse = __shfl(logs, 0), lse0 = __shfl(logs, 1) + ((empty ? 0.0 : R) - whole_r);
        const double log_q0 = __shfl(logs, 2), log_sum = tail ? 0 : __shfl(logs, 3);
        const double a_mass = mass + q0;
        double loss = 0;
#pragma unroll 1
        for (uint32_t j = lane; j < k; j += kLanes) {
            double grad = 0;
            if (col[j] >= 0) {
                const double qj = q[j] * scale, arg = times(sl[j], cd) - whole_r - lse;
                const bool zero = sl[j] == -INFINITY;
                if (qj > 0)
                    loss += zero ? INFINITY
                                 : qj * (static_cast<double>(tl[j]) * a.inv_t - known - (log_sum + arg) * kLn2);
                double all = q[j];  // what the teacher puts on this column, if it is there more than once
                if (*again) {
                    all = 0;
#pragma unroll 1
                    for (uint32_t i = 0; i < k; ++i)
                        if (col[i] == col[j]) all += q[i];
                }
                grad = (zero ? 0 : a_mass * power_of_two(arg)) - all * scale;
            }
            const float gj = static_cast<float>(grad);
            if (stats) stats[kStats + j] = gj;
            sl[j] = gj;
        }
        loss = wave_sum(loss);
        if (lane == 0) {
            if (q0 > 0) loss += empty ? INFINITY : q0 * (log_q0 - (lse0 - lse)) * kLn2;
            a.row_loss[row] = static_cast<float>(loss);
            double f = 0;
            if (!empty) {
                f = a_mass * scaled(1.0, R - whole_r) / whole;
                if (q0 > 0) f -= q0 / z;
            }
            out[0] = empty ? 0.0 : R;
            out[1] = f;
            *base = base_of(out[0], cd);
            if (stats) write_stats(stats, out[0], *base, f);
        }
    }
    if constexpr (GRAD) {
        __syncthreads();
        const float scale = weight * static_cast<float>(a.inv_t), f = static_cast<float>(out[1]) * scale;
        const float from = *base;
        r = from != 0.f || reference == -INFINITY ? 0.f : static_cast<float>(out[0]);
        // 16-bit gradients: the factor joins the exponent, where that keeps it to
        // 2^-19, and its sign the result
        const float joint = r - __builtin_amdgcn_logf(fabsf(f));
        if (T != kRowF32 && fabsf(joint) < 64.f) {
            r = joint;
            sign = f < 0.f ? 0x80008000u : 0u;
        } else {
            factor = f;
        }
#pragma unroll
        for (int u = 0; u < V; ++u) {
            if (below(vecs, u)) {
                float e[kVec];
                unpack16<T>(v[u], e);
                if (from != 0.f) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) e[i] -= from;
                }
#pragma unroll
                for (int i = 0; i < kVec; ++i) e[i] = __builtin_amdgcn_exp2f(exponent<T>(e[i], c, a.c_low, r));
                if (factor != 1.f) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) e[i] *= factor;
                }
                u32x4 w = pack16<T>(e);
                if (T != kRowF32) w ^= sign;
                store16_once(reinterpret_cast<uint8_t *>(g + u * B * kVec) + tid * 16, w);
            }
        }
        if (rest < n) {
            const float e = __builtin_amdgcn_exp2f(exponent<T>(over - from, c, a.c_low, r));
            g[rest] = Row<T>::pattern(e * factor) ^ static_cast<Stored>(sign);
        }
        // the teacher's columns over what was written there
        __syncthreads();
#pragma unroll 1
        for (uint32_t j = tid; j < k; j += B)
            if (col[j] >= 0) g[col[j]] = Row<T>::pattern(sl[j] * scale);
    }
}

// How many workgroups share a row: enough that few rows still fill the GPU,
// each with a piece worth a workgroup.
void distill_split(uint64_t rows, uint64_t n, uint32_t &splits, uint32_t &len) {
    uint64_t s = 1;
    if (rows < 2048) s = std::min<uint64_t>((2048 + rows - 1) / std::max<uint64_t>(rows, 1), n / 8192);
    s = std::max<uint64_t>(1, s);
    const uint64_t l = std::max<uint64_t>(8, ((n + s - 1) / s + 7) / 8 * 8);
    len = static_cast<uint32_t>(l);
    splits = static_cast<uint32_t>(std::max<uint64_t>(1, (n + l - 1) / l));
}

int check_sizes(int64_t rows, int64_t n, int64_t k, int dtype) {
    if (!row_type_ok(dtype)) return LRS_ERR_DTYPE;
    if (rows < 0 || n < 0 || k < 1 || k > LRS_MAX_TOPK || static_cast<uint64_t>(n) > LRS_MAX_ROW_LEN) return LRS_ERR_SIZE;
    if (static_cast<uint64_t>(rows) >= (uint64_t(1) << 40) / std::max<uint64_t>(1, static_cast<uint64_t>(n)))
        return LRS_ERR_SIZE;
    return LRS_OK;
}
struct DisSpace {
    uint64_t partial = 0, stats = 0, row_loss = 0, total = 0;
};
DisSpace distill_space(uint64_t rows, uint64_t n, uint64_t k) {
    DisSpace w;
    if (rows == 0) return w;
    uint32_t splits, len;
    distill_split(rows, n, splits, len);
    auto place = [&](uint64_t bytes) {
        const uint64_t at = w.total;
        w.total += (bytes + 255) / 256 * 256;
        return at;
    };
    // the same whichever form the rows take
    w.partial = place(rows * splits * sizeof(Partial));
    w.stats = place(rows * (k + kStats) * sizeof(float));
    w.row_loss = place(rows * sizeof(float));
    return w;
}

// Everything the three calls check of the inputs; fills the arguments.
int distill_inputs(const lrs_distill *d, DisArgs &a) {
    if (d == nullptr) return LRS_ERR_NULL_POINTER;
    const int st = check_sizes(d->rows, d->n, d->k, d->dtype);
    if (st != LRS_OK) return st;
    if (!row_type_ok(d->teacher_dtype) || (d->index_bytes != 4 && d->index_bytes != 8)) return LRS_ERR_DTYPE;
    if (!stride_ok(d->row_stride, d->rows) || !stride_ok(d->teacher_stride, d->rows) || !stride_ok(d->index_stride, d->rows))
        return LRS_ERR_SIZE;
    if (!(d->temperature > 0) || !std::isfinite(d->temperature) || !std::isfinite(static_cast<float>(kLog2e / d->temperature)))
        return LRS_ERR_OPTION;
    if (d->rows > 0 && ((d->n > 0 && !d->logits) || !d->teacher_values || !d->teacher_indices))
        return LRS_ERR_NULL_POINTER;
    if (misaligned(d->logits, row_type_size(d->dtype)) || misaligned(d->teacher_values, row_type_size(d->teacher_dtype)) ||
        misaligned(d->teacher_indices, d->index_bytes) || misaligned(d->teacher_lse, 4) || misaligned(d->row_weights, 4))
        return LRS_ERR_ALIGNMENT;
    a.logits = d->logits;
    a.stride = d->row_stride;
    a.rows = d->rows;
    a.n = static_cast<uint32_t>(d->n);
    a.k = static_cast<uint32_t>(d->k);
    a.tv = d->teacher_values;
    a.tv_stride = d->teacher_stride;
    a.tv_type = d->teacher_dtype;
    a.ti = d->teacher_indices;
    a.ti_stride = d->index_stride;
    a.ti_bytes = d->index_bytes;
    a.tlse = d->teacher_lse;
    a.weights = d->row_weights;
    a.inv_t = 1.0 / d->temperature;
    const double factor = kLog2e * a.inv_t;
    // both parts above 0, so that -inf times either is -inf: the first is rounded
    // down, and neither is below the smallest number (times the largest: 2^-21)
    constexpr float kLeast = std::numeric_limits<float>::denorm_min();
    a.c = static_cast<float>(factor);
    if (a.c > factor) a.c = std::nextafter(a.c, 0.f);
    a.c = std::max(a.c, kLeast);
    a.c_low = std::max(static_cast<float>(factor - a.c), kLeast);
    distill_split(a.rows, a.n, a.splits, a.split_len);
    return LRS_OK;
}

// Whether [p, p + bytes) touches any input.
bool hits_input(const lrs_distill *d, const void *p, uint64_t bytes) {
    const uint64_t r = d->rows, k = d->k;
    return overlaps(p, bytes, d->logits, span(r, d->row_stride, d->n, row_type_size(d->dtype))) ||
           overlaps(p, bytes, d->teacher_values, span(r, d->teacher_stride, k, row_type_size(d->teacher_dtype))) ||
           overlaps(p, bytes, d->teacher_indices, span(r, d->index_stride, k, d->index_bytes)) ||
           overlaps(p, bytes, d->teacher_lse, d->teacher_lse ? 4 * r : 0) ||
           overlaps(p, bytes, d->row_weights, d->row_weights ? 4 * r : 0);
}

constexpr uint64_t kMaxGrid = 1u << 20;

template <int T> void distill_launch_sums(const DisArgs &a, const Ctx &c) {
    const dim3 grid(static_cast<uint32_t>(std::min<uint64_t>(a.rows * a.splits, kMaxGrid)));
    {
        TimedLaunch t(4, c);
        if (a.tlse != nullptr)
            launch_on(distill_sum_kernel<T, true>, grid, dim3(kDisBlock), t.L, a);
        else
            launch_on(distill_sum_kernel<T, false>, grid, dim3(kDisBlock), t.L, a);
    }
    TimedLaunch t(4, c);
    launch_on(distill_row_kernel<T>, dim3(static_cast<uint32_t>(std::min<uint64_t>(a.rows, kMaxGrid))), dim3(kLanes), t.L, a);
}

template <int T> void distill_launch_grad(const DisArgs &a, const Ctx &c) {
    TimedLaunch t(4, c);
    launch_on(distill_grad_kernel<T>, dim3(static_cast<uint32_t>(std::min<uint64_t>(a.rows * a.splits, kMaxGrid))),
              dim3(kDisBlock), t.L, a);
}

// Rows of at most 256 KB are held in registers: by workgroups of 1024 threads
// where there are no more rows than CUs, by the fewest threads that hold one
// where several workgroups share a CU.
constexpr uint64_t kHeldBytes = 1024 * 16 * 16;
bool distill_held(uint64_t n, uint64_t size) { return n * size <= kHeldBytes; }

template <int T> void distill_launch_held(const DisArgs &a, uint32_t rows, const Ctx &c) {
    TimedLaunch t(4, c);
    const uint32_t lds = HeldLds::bytes(a.k, a.n);
    const uint64_t vecs = a.n / Row<T>::kVec;
    const auto go = [&](auto grad, auto loss, int block) {
        launch_lds(a.grad ? grad : loss, dim3(rows), dim3(block), lds, t.L, a);
    };
    if (a.rows <= 256) {
        if (vecs <= 1024 * 2) return go(distill_held_kernel<T, 1024, 2, true>, distill_held_kernel<T, 1024, 2, false>, 1024);
        if (vecs <= 1024 * 4) return go(distill_held_kernel<T, 1024, 4, true>, distill_held_kernel<T, 1024, 4, false>, 1024);
        if (vecs <= 1024 * 8) return go(distill_held_kernel<T, 1024, 8, true>, distill_held_kernel<T, 1024, 8, false>, 1024);
        return go(distill_held_kernel<T, 1024, 16, true>, distill_held_kernel<T, 1024, 16, false>, 1024);
    }
    // a wave for up to 8 KB, so that many short rows' chains run side by side
    // (8192 x 600 bf16 step: 20 us, 36 us by workgroups of 256)
    if (vecs <= 64 * 4) return go(distill_held_kernel<T, 64, 4, true>, distill_held_kernel<T, 64, 4, false>, 64);
    if (vecs <= 64 * 8) return go(distill_held_kernel<T, 64, 8, true>, distill_held_kernel<T, 64, 8, false>, 64);
    if (vecs <= 128 * 8) return go(distill_held_kernel<T, 128, 8, true>, distill_held_kernel<T, 128, 8, false>, 128);
    if (vecs <= 256 * 8) return go(distill_held_kernel<T, 256, 8, true>, distill_held_kernel<T, 256, 8, false>, 256);
    if (vecs <= 256 * 16) return go(distill_held_kernel<T, 256, 16, true>, distill_held_kernel<T, 256, 16, false>, 256);
    if (vecs <= 512 * 16) return go(distill_held_kernel<T, 512, 16, true>, distill_held_kernel<T, 512, 16, false>, 512);
    go(distill_held_kernel<T, 1024, 16, true>, distill_held_kernel<T, 1024, 16, false>, 1024);
}

// The loss and what a gradient needs; with a.grad and held rows the gradient too.
int distill_forward(const DisArgs &a, int dtype, const Ctx &c) {
    if (a.rows > 0 && distill_held(a.n, row_type_size(dtype))) {
        DisArgs part = a;
        for (; part.first_row < a.rows; part.first_row += kMaxGrid) {
            const uint32_t rows = static_cast<uint32_t>(std::min<uint64_t>(a.rows - part.first_row, kMaxGrid));
            if (dtype == LRS_DTYPE_FP16) distill_launch_held<kRowF16>(part, rows, c);
            else if (dtype == LRS_DTYPE_BF16) distill_launch_held<kRowBF16>(part, rows, c);
            else distill_launch_held<kRowF32>(part, rows, c);
            if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
        }
    } else if (a.rows > 0) {
        if (dtype == LRS_DTYPE_FP16) distill_launch_sums<kRowF16>(a, c);
        else if (dtype == LRS_DTYPE_BF16) distill_launch_sums<kRowBF16>(a, c);
        else distill_launch_sums<kRowF32>(a, c);
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
    }
    TimedLaunch t(4, c);
    launch_on(distill_loss_kernel, dim3(1), dim3(1024), t.L, a);
    return hipGetLastError() == hipSuccess ? LRS_OK : LRS_ERR_HIP;
}

int distill_backward(const DisArgs &a, int dtype, const Ctx &c) {
    if (a.rows == 0 || a.n == 0) return LRS_OK;
    if (dtype == LRS_DTYPE_FP16) distill_launch_grad<kRowF16>(a, c);
    else if (dtype == LRS_DTYPE_BF16) distill_launch_grad<kRowBF16>(a, c);
    else distill_launch_grad<kRowF32>(a, c);
    return hipGetLastError() == hipSuccess ? LRS_OK : LRS_ERR_HIP;
}

// Forward with or without a gradient.
int distill_run(const lrs_distill *d, float *loss, float *row_loss, float *stats, void *grad, int64_t grad_stride,
                bool step, void *workspace, size_t workspace_bytes, void *stream, const lrs_options *opts) {
    Ctx c;
    if (!make_ctx(stream, opts, c)) return LRS_ERR_OPTION;
    DisArgs a{};
    const int st = distill_inputs(d, a);
    if (st != LRS_OK) return st;
    if (step && (!stride_ok(grad_stride, d->rows) || (d->rows > 1 && grad_stride < d->n))) return LRS_ERR_SIZE;
    const DisSpace w = distill_space(a.rows, a.n, a.k);
    if (!loss || (w.total && !workspace) || (step && a.rows && a.n && !grad)) return LRS_ERR_NULL_POINTER;
    const uint64_t size = row_type_size(d->dtype);
    if (misaligned(loss, 4) || misaligned(row_loss, 4) || misaligned(stats, 4) || misaligned(grad, size) ||
        (w.total && misaligned(workspace, 256)))
        return LRS_ERR_ALIGNMENT;
    if (workspace_bytes < w.total) return LRS_ERR_WORKSPACE_TOO_SMALL;
    const uint64_t lb = row_loss ? 4 * a.rows : 0, sb = stats ? 4 * a.rows * (a.k + kStats) : 0;
    const uint64_t gb = step ? span(a.rows, grad_stride, a.n, size) : 0;
    const void *out[] = {loss, row_loss, stats, grad, workspace};
    const uint64_t bytes[] = {4, lb, sb, gb, w.total};
    for (int i = 0; i < 5; ++i) {
        if (bytes[i] == 0) continue;
        if (hits_input(d, out[i], bytes[i])) return LRS_ERR_ALIASING;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], bytes[i], out[j], bytes[j])) return LRS_ERR_ALIASING;
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.partial = reinterpret_cast<Partial *>(ws + w.partial);
    const bool held = distill_held(a.n, size);
    a.stats = stats || held ? stats : reinterpret_cast<float *>(ws + w.stats);
    a.row_loss = row_loss ? row_loss : reinterpret_cast<float *>(ws + w.row_loss);
    a.loss = loss;
    a.grad = grad;
    a.grad_stride = static_cast<uint64_t>(grad_stride);
    c.elems = a.rows * a.n;
    const int fs = distill_forward(a, d->dtype, c);
    return fs != LRS_OK || !step || held ? fs : distill_backward(a, d->dtype, c);
}

}  // namespace
}  // namespace lrs

using namespace lrs;

extern "C" {

size_t topk_distill_workspace_size(int64_t rows, int64_t n, int64_t k, int dtype, const lrs_options *opts) {
    if (!options_ok(opts) || check_sizes(rows, n, k, dtype) != LRS_OK) return 0;
    return static_cast<size_t>(distill_space(rows, n, k).total);
}

int topk_distill_forward(const lrs_distill *in, float *loss, float *row_loss, float *row_stats, void *workspace,
                         size_t workspace_bytes, void *stream, const lrs_options *opts) try {
    return distill_run(in, loss, row_loss, row_stats, nullptr, 0, false, workspace, workspace_bytes, stream, opts);
} catch (...) {
    return LRS_ERR_HIP;
}

int topk_distill_step(const lrs_distill *in, float *loss, float *row_loss, void *grad, int64_t grad_stride,
                      void *workspace, size_t workspace_bytes, void *stream, const lrs_options *opts) try {
    return distill_run(in, loss, row_loss, nullptr, grad, grad_stride, true, workspace, workspace_bytes, stream, opts);
} catch (...) {
    return LRS_ERR_HIP;
}

int topk_distill_backward(const lrs_distill *in, const float *row_stats, const float *loss_grad, void *grad,
                          int64_t grad_stride, void *stream, const lrs_options *opts) try {
    Ctx c;
    if (!make_ctx(stream, opts, c)) return LRS_ERR_OPTION;
    DisArgs a{};
    const int st = distill_inputs(in, a);
    if (st != LRS_OK) return st;
    if (!stride_ok(grad_stride, in->rows) || (in->rows > 1 && grad_stride < in->n)) return LRS_ERR_SIZE;
    if (a.rows == 0 || a.n == 0) return LRS_OK;
    if (!row_stats || !grad) return LRS_ERR_NULL_POINTER;
    const uint64_t size = row_type_size(in->dtype);
    if (misaligned(row_stats, 4) || misaligned(loss_grad, 4) || misaligned(grad, size)) return LRS_ERR_ALIGNMENT;
    const uint64_t gb = span(a.rows, grad_stride, a.n, size);
    if (hits_input(in, grad, gb) || overlaps(grad, gb, row_stats, 4 * a.rows * (a.k + kStats)) ||
        overlaps(grad, gb, loss_grad, loss_grad ? 4 : 0))
        return LRS_ERR_ALIASING;
    a.stats = const_cast<float *>(row_stats);
    a.loss_grad = loss_grad;
    a.grad = grad;
    a.grad_stride = static_cast<uint64_t>(grad_stride);
    c.elems = a.rows * a.n;
    return distill_backward(a, in->dtype, c);
} catch (...) {
    return LRS_ERR_HIP;
}

}  // extern "C"
