// sequences.h -- packed sequences for the Mamba-2 operators over many tokens (gfx950), private to the library.
//
// S sequences lie one after another in T rows: sequence s in rows [cu[s], cu[s + 1]), or, without
// offsets, S sequences of T / S rows each.  Offsets live in device memory, so the host cannot check them; every reader
// cuts them to [0, T], which keeps bad ones inside the buffers (what they compute is then unspecified).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"

namespace dfssm {

struct Sequences {
    const int32_t* cu;  // [S + 1], or NULL
    int T, S, L;        // L: the common length without offsets
};

struct Span {
    int begin, end;
};

__device__ __forceinline__ Span span_of(const Sequences& q, int s) {
    if (!q.cu) return {s * q.L, (s + 1) * q.L};
    int b = q.cu[s], e = q.cu[s + 1];
    b = b < 0 ? 0 : b > q.T ? q.T : b;
    e = e < b ? b : e > q.T ? q.T : e;
    return {b, e};
}

// The last sequence that starts at row t or before it (rows before the first one: sequence 0, whose span excludes them).
__device__ __forceinline__ int sequence_at(const Sequences& q, int t) {
    if (!q.cu) return t / q.L;
    int lo = 0, hi = q.S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (q.cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Elements of either type as fp32, one or four at a time.
template <bool kBf16>
struct Elem;
template <>
struct Elem<false> {
    using type = float;
    static __device__ __forceinline__ float load(const float* p) { return *p; }
    static __device__ __forceinline__ v4f load4(const float* p) { return *reinterpret_cast<const v4f*>(p); }
    static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
    static __device__ __forceinline__ void store4(float* p, v4f v) { *reinterpret_cast<v4f*>(p) = v; }
};
template <>
struct Elem<true> {
    using type = uint16_t;
    static __device__ __forceinline__ float load(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
    static __device__ __forceinline__ v4f load4(const uint16_t* p) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        return {__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                __uint_as_float(v.y & 0xFFFF0000u)};
    }
    static __device__ __forceinline__ void store(uint16_t* p, float v) { *p = (uint16_t)bf16_bits(v); }
    static __device__ __forceinline__ void store4(uint16_t* p, v4f v) {
        *reinterpret_cast<uint2*>(p) =
            make_uint2(bf16_bits(v.x) | (bf16_bits(v.y) << 16), bf16_bits(v.z) | (bf16_bits(v.w) << 16));
    }
};

// A chunk's rows of a matrix, from column `col` on, as a buffer: what lies past the last row's `width` elements reads as zero and
// is not written, so rows behind a sequence need no branch, and offsets are 32 bits (row strides of up to 2^22 elements).
template <bool kBf16>
struct RowBuffer {
    __amdgpu_buffer_rsrc_t rsrc;
    static constexpr int kSize = kBf16 ? 2 : 4;
    __device__ __forceinline__ RowBuffer(const void* base, int64_t first, int64_t ld, int rows, int64_t col, int width)
        : rsrc(make_rsrc(static_cast<const uint8_t*>(base) + (first * ld + col) * kSize,
                         (uint32_t)(((rows - 1) * (uint32_t)ld + (uint32_t)width) * kSize))) {}
    __device__ __forceinline__ float load(int bytes) const {
        if constexpr (kBf16) return __uint_as_float((uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rsrc, bytes, 0, 0) << 16);
        else return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsrc, bytes, 0, 0));
    }
    __device__ __forceinline__ v4f load4(int bytes) const {
        if constexpr (kBf16) {
            const auto v = __builtin_amdgcn_raw_buffer_load_b64(rsrc, bytes, 0, 0);
            return {__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xFFFF0000u), __uint_as_float(v[1] << 16),
                    __uint_as_float(v[1] & 0xFFFF0000u)};
        } else {
            return __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rsrc, bytes, 0, 0));
        }
    }
    // two neighbours (an even place), as they lie in memory
    using Pair = std::conditional_t<kBf16, uint32_t, uint64_t>;
    __device__ __forceinline__ Pair load2(int bytes) const {
        if constexpr (kBf16) return __builtin_amdgcn_raw_buffer_load_b32(rsrc, bytes, 0, 0);
        else return __builtin_bit_cast(uint64_t, __builtin_amdgcn_raw_buffer_load_b64(rsrc, bytes, 0, 0));
    }
    static __device__ __forceinline__ float first(Pair v) {
        if constexpr (kBf16) return __uint_as_float(v << 16);
        else return __uint_as_float((uint32_t)v);
    }
    static __device__ __forceinline__ float second(Pair v) {
        if constexpr (kBf16) return __uint_as_float(v & 0xFFFF0000u);
        else return __uint_as_float((uint32_t)(v >> 32));
    }
    __device__ __forceinline__ void store2(float x, float y, int bytes) const {
        if constexpr (kBf16) {
            __builtin_amdgcn_raw_buffer_store_b32(bf16_bits(x) | (bf16_bits(y) << 16), rsrc, bytes, 0, 0);
        } else {
            typedef uint32_t v2u __attribute__((ext_vector_type(2)));
            __builtin_amdgcn_raw_buffer_store_b64(v2u{__float_as_uint(x), __float_as_uint(y)}, rsrc, bytes, 0, 0);
        }
    }
    __device__ __forceinline__ void store(float v, int bytes) const {
        if constexpr (kBf16) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)bf16_bits(v), rsrc, bytes, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rsrc, bytes, 0, 0);
    }
};

// A lane's offset that the optimizer takes as new: what is computed from it is not kept in registers from one turn of a loop
// to the next (an empty asm statement emits no instruction).
__device__ __forceinline__ int opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

}  // namespace dfssm
