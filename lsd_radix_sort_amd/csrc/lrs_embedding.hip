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
    const uint32_t *sorted, *sorted_places;
};

// The keys of the sort: ids, those that count for nothing behind the last.
__global__ __launch_bounds__(kEmbBlock) void embed_keys_kernel(GradArgs a) {
    const uint32_t t = blockIdx.x * kEmbBlock + threadIdx.x;
    if (t >= a.tokens) return;
    const int64_t id = a.ids[t];
    a.keys[t] = id >= 0 && id < a.vocab && id != a.padding ? static_cast<uint32_t>(id) : a.vocab;
    a.places[t] = t;
}

__device__ inline uint32_t first_of(const uint32_t *keys, uint32_t count, uint32_t id) {
    uint32_t lo = 0, hi = count;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (keys[mid] < id) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

template <int T, int O>
__global__ __launch_bounds__(kEmbBlock) void embed_sum_kernel(GradArgs a) {
    for (uint32_t v = blockIdx.x; v < a.vocab; v += gridDim.x) {
        const uint32_t from = first_of(a.sorted, a.tokens, v), to = first_of(a.sorted, a.tokens, v + 1);
        if (a.accumulate && from == to) continue;
        for (uint32_t first = threadIdx.x * 8; first < a.width; first += kEmbBlock * 8) {
            const bool whole = first + 8 <= a.width;
            const uint32_t n = whole ? 8 : a.width - first;
            float sum[8] = {};
            for (uint32_t i = from; i < to; ++i) {
                const uint64_t at = a.sorted_places[i] * a.grad_stride + first;
                float f[8] = {};
                if (whole) load8<T>(a.grad, at, f);
                else
                    for (uint32_t e = 0; e < n; ++e) f[e] = Row<T>::value(static_cast<const typename Row<T>::Stored *>(a.grad)[at + e]);
                for (int e = 0; e < 8; ++e) sum[e] += f[e];
            }
            auto *out = static_cast<typename Row<O>::Stored *>(a.out) + v * a.out_stride + first;
            for (uint32_t e = 0; e < n; ++e) {
                const float old = a.accumulate ? Row<O>::value(out[e]) : 0.f;
                out[e] = Row<O>::pattern(fmaf(sum[e], a.scale, old));
            }
        }
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

struct GradSpace {
    uint64_t keys = 0, places = 0, sorted = 0, sorted_places = 0, sort = 0, sort_bytes = 0, total = 0;
};
int key_bits(uint64_t vocab) {
    int b = 1;
    while ((vocab >> b) != 0) ++b;  // keys are at most vocab
    return b;
}
GradSpace grad_space(uint64_t tokens, uint64_t vocab, const lrs_options *opts) {
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
    w.sorted_places = place(4 * tokens);
    w.sort_bytes = radix_sort_workspace_size(tokens, 0, key_bits(vocab), 8, 1, opts);
    w.sort = place(w.sort_bytes);
    return w;
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
    return static_cast<size_t>(grad_space(tokens, vocab, opts).total);
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
    const GradSpace w = grad_space(count, vocab, opts);
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
    if (count > 0) {
        uint8_t *ws = static_cast<uint8_t *>(workspace);
        a.keys = reinterpret_cast<uint32_t *>(ws + w.keys);
        a.places = reinterpret_cast<uint32_t *>(ws + w.places);
        uint32_t *sorted = reinterpret_cast<uint32_t *>(ws + w.sorted), *order = reinterpret_cast<uint32_t *>(ws + w.sorted_places);
        a.sorted = sorted;
        a.sorted_places = order;
        {
            TimedLaunch t(4, c);
            launch_on(embed_keys_kernel, dim3((a.tokens + kEmbBlock - 1) / kEmbBlock), dim3(kEmbBlock), t.L, a);
        }
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
        st = radix_sort_pairs(a.keys, a.places, sorted, order, a.tokens, 0, key_bits(vocab), 8, ws + w.sort, w.sort_bytes,
                              stream, opts);
        if (st != LRS_OK) return st;
    }
    TimedLaunch t(4, c);
    const dim3 grid(static_cast<uint32_t>(std::min<uint64_t>(vocab, kMaxGrid)));
    by_types(dtype, out_dtype, [&](auto i, auto o) { launch_on(embed_sum_kernel<i.value, o.value>, grid, dim3(kEmbBlock), t.L, a); });
    return hipGetLastError() == hipSuccess ? LRS_OK : LRS_ERR_HIP;
} catch (...) {
    return LRS_ERR_HIP;
}

}  // extern "C"
