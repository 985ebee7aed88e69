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

// For what is read or written once: the same, without keeping it in the caches.
__device__ inline u32x4 load16_once(const void *p) {
    return __builtin_nontemporal_load(static_cast<const u32x4_align2 *>(p));
}
__device__ inline void store16_once(void *p, u32x4 v) {
    __builtin_nontemporal_store(v, static_cast<u32x4_align2 *>(p));
}

// The task of a workgroup where each XCD takes a contiguous share of them
// (workgroups go to the 8 XCDs in turn).
__device__ inline uint32_t xcd_chunk(uint32_t block, uint32_t blocks) {
    const uint32_t xcd = block % 8, share = blocks / 8, more = blocks % 8;
    return xcd * share + min(xcd, more) + block / 8;
}

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

// The lanes' values moved by a DPP control; lanes without a source, and rows of
// 16 lanes outside ROWS, get `none`.
template <int CONTROL, int ROWS = 0xF, typename V> __device__ inline V moved(V v, V none) {
    static_assert(sizeof(V) == 4 || sizeof(V) == 8);
    if constexpr (sizeof(V) == 4) {
        return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v),
                                                                 CONTROL, ROWS, 0xF, false));
    } else {
        typedef int pair __attribute__((ext_vector_type(2)));
        const pair p = __builtin_bit_cast(pair, v), o = __builtin_bit_cast(pair, none);
        const pair r = {__builtin_amdgcn_update_dpp(o.x, p.x, CONTROL, ROWS, 0xF, false),
                        __builtin_amdgcn_update_dpp(o.y, p.y, CONTROL, ROWS, 0xF, false)};
        return __builtin_bit_cast(V, r);
    }
}
template <typename V> __device__ inline V last_lane(V v) {
    if constexpr (sizeof(V) == 4) {
        return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), kLanes - 1));
    } else {
        typedef int pair __attribute__((ext_vector_type(2)));
        const pair p = __builtin_bit_cast(pair, v);
        const pair r = {__builtin_amdgcn_readlane(p.x, kLanes - 1), __builtin_amdgcn_readlane(p.y, kLanes - 1)};
        return __builtin_bit_cast(V, r);
    }
}
// Joins the values of a whole wave, every lane active, in a fixed order: within
// rows of 16 lanes (row_shr 1, 2, 4, 8), then across them (row_bcast 15, 31).
// The result is the same in every lane, in scalar registers.
template <typename V, typename F> __device__ inline V wave_join(V v, V none, F join) {
    v = join(v, moved<0x111>(v, none));
    v = join(v, moved<0x112>(v, none));
    v = join(v, moved<0x114>(v, none));
    v = join(v, moved<0x118>(v, none));
    v = join(v, moved<0x142, 0xA>(v, none));
    v = join(v, moved<0x143, 0xC>(v, none));
    return last_lane(v);
}
// Sums and the largest of every `lanes` neighbours of a wave (a power of two), in
// each of them: quads, eights and sixteens by quad_perm, row_half_mirror and
// row_mirror, then across rows.
template <int CONTROL> __device__ inline float swapped(float v) {  // every lane has a source: joins with what uses it
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CONTROL, 0xF, 0xF, true));
}
// The largest of three, without the instructions that would quiet a signalling NaN first.
__device__ inline float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ inline float2 group_join(float2 v, uint32_t lanes) {
    const auto add = [&](float p, float q) {
        v.x += p;
        v.y += q;
    };
    if (lanes > 1) add(swapped<0xB1>(v.x), swapped<0xB1>(v.y));
    if (lanes > 2) add(swapped<0x4E>(v.x), swapped<0x4E>(v.y));
    if (lanes > 4) add(swapped<0x141>(v.x), swapped<0x141>(v.y));
    if (lanes > 8) add(swapped<0x140>(v.x), swapped<0x140>(v.y));
    if (lanes > 16) add(__shfl_xor(v.x, 16), __shfl_xor(v.y, 16));
    if (lanes > 32) add(__shfl_xor(v.x, 32), __shfl_xor(v.y, 32));
    return v;
}
__device__ inline float group_max(float v, uint32_t lanes) {
    const auto join = [&](float p) { v = max3(v, p, p); };
    if (lanes > 1) join(swapped<0xB1>(v));
    if (lanes > 2) join(swapped<0x4E>(v));
    if (lanes > 4) join(swapped<0x141>(v));
    if (lanes > 8) join(swapped<0x140>(v));
    if (lanes > 16) join(__shfl_xor(v, 16));
    if (lanes > 32) join(__shfl_xor(v, 32));
    return v;
}
template <typename V> __device__ inline V wave_sum(V v) {
    return wave_join(v, V(0), [](V a, V b) { return a + b; });
}
__device__ inline float wave_max(float v) {
    return wave_join(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}
__device__ inline double wave_max(double v) {
    return wave_join(v, static_cast<double>(-INFINITY), [](double a, double b) { return fmax(a, b); });
}

}  // namespace lrs
