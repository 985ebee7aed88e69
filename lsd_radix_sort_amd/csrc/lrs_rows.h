// lrs_rows.h -- device helpers of the row operators (internal header): element
// types, 16-byte loads and stores at any element alignment, wave reductions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lrs {

constexpr int kLanes = 64;  // CDNA wavefront width

// Row element types, numbered as LRS_DTYPE_*.
enum RowType : int { kRowF16 = 0, kRowBF16 = 1, kRowF32 = 2 };

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Sixteen bytes at the alignment of one element.  Rows of odd strides start at
// any element; one global_load_dwordx4 per lane at any byte address costs a
// wave one more cache line than the aligned load.
typedef u32x4 u32x4_align2 __attribute__((aligned(2)));
__device__ inline u32x4 load16(const void *p) { return *static_cast<const u32x4_align2 *>(p); }
__device__ inline void store16(void *p, u32x4 v) { *static_cast<u32x4_align2 *>(p) = v; }

template <int T> struct Row;

template <> struct Row<kRowF16> {
    using Stored = uint16_t;
    static constexpr int kVec = 8;  // elements in 16 bytes
    __device__ static inline float value(uint16_t v) { return static_cast<float>(__builtin_bit_cast(_Float16, v)); }
    __device__ static inline uint16_t pattern(float f) {
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
    }
    __device__ static inline void unpack(uint32_t w, float &a, float &b) {
        const f16x2 h = __builtin_bit_cast(f16x2, w);
        a = static_cast<float>(h.x);
        b = static_cast<float>(h.y);
    }
    __device__ static inline uint32_t pack(float a, float b) {
        const f32x2 f = {a, b};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
    }
};

template <> struct Row<kRowBF16> {
    using Stored = uint16_t;
    static constexpr int kVec = 8;
    __device__ static inline float value(uint16_t v) {
        return __builtin_bit_cast(float, static_cast<uint32_t>(v) << 16);
    }
    __device__ static inline uint16_t pattern(float f) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f)); }
    __device__ static inline void unpack(uint32_t w, float &a, float &b) {
        a = __builtin_bit_cast(float, w << 16);
        b = __builtin_bit_cast(float, w & 0xFFFF0000u);
    }
    __device__ static inline uint32_t pack(float a, float b) {
        const f32x2 f = {a, b};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
    }
};

template <> struct Row<kRowF32> {
    using Stored = uint32_t;
    static constexpr int kVec = 4;
    __device__ static inline float value(uint32_t v) { return __builtin_bit_cast(float, v); }
    __device__ static inline uint32_t pattern(float f) { return __builtin_bit_cast(uint32_t, f); }
};

// The kVec elements of a 16-byte word as floats, and back.
template <int T> __device__ inline void unpack16(u32x4 v, float (&f)[Row<T>::kVec]) {
    if constexpr (T == kRowF32) {
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = v[i];  // a bit cast of v[i] itself reads element 0 here
            f[i] = __builtin_bit_cast(float, w);
        }
    } else {
        for (int i = 0; i < 4; ++i) Row<T>::unpack(v[i], f[2 * i], f[2 * i + 1]);
    }
}
template <int T> __device__ inline u32x4 pack16(const float (&f)[Row<T>::kVec]) {
    u32x4 v;
    if constexpr (T == kRowF32) {
        for (int i = 0; i < 4; ++i) v[i] = __builtin_bit_cast(uint32_t, f[i]);
    } else {
        for (int i = 0; i < 4; ++i) v[i] = Row<T>::pack(f[2 * i], f[2 * i + 1]);
    }
    return v;
}

template <typename V> __device__ inline V wave_sum(V v) {
    for (int d = kLanes / 2; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
__device__ inline float wave_max(float v) {
    for (int d = kLanes / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
__device__ inline double wave_max(double v) {
    for (int d = kLanes / 2; d > 0; d >>= 1) v = fmax(v, __shfl_xor(v, d));
    return v;
}

}  // namespace lrs
