// storage.cuh -- tensors stored as binary32, binary16 or bfloat16 (REPOPS_TYPE_*)
// around binary32 arithmetic: exact widening on load, one rounding to nearest
// even on store; and the spans of pitched rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.cuh"

namespace repops {
namespace {

[[maybe_unused]] inline bool known_storage(int t) {
    return t == REPOPS_TYPE_F32 || t == REPOPS_TYPE_F16 || t == REPOPS_TYPE_BF16;
}
[[maybe_unused]] inline unsigned storage_size(int t) { return t == REPOPS_TYPE_F32 ? 4u : 2u; }

// Whether an address is no multiple of `size` bytes (null is).
[[maybe_unused]] inline bool misaligned(const void *p, unsigned size) { return reinterpret_cast<uintptr_t>(p) % size != 0; }

// Bytes spanned by rows x cols elements of `size` bytes at pitch ld; false
// when ld is short or the span overflows.
[[maybe_unused]] inline bool span_bytes(int64_t rows, int64_t cols, int64_t ld, unsigned size, uint64_t *bytes) {
    *bytes = 0;
    if (ld < cols) return false;
    if (rows == 0 || cols == 0) return true;
    if (ld > INT64_MAX / 8 || rows - 1 > (INT64_MAX / 8 - cols) / ld) return false;
    *bytes = uint64_t((rows - 1) * ld + cols) * size;
    return true;
}

template <int TY>
__device__ __forceinline__ float load_one(const DbgAccess &d, const void *p, int64_t i) {
    if constexpr (TY == REPOPS_TYPE_F32) return load_global(d, static_cast<const float *>(p) + i);
    else if constexpr (TY == REPOPS_TYPE_F16) return __half2float(load_global(d, static_cast<const __half *>(p) + i));
    else return __bfloat162float(load_global(d, static_cast<const __nv_bfloat16 *>(p) + i));
}

// A value as it is stored: 32 bits, or 16 in the low half.
template <int TY>
__device__ __forceinline__ uint32_t narrowed(float v) {
    if constexpr (TY == REPOPS_TYPE_F32) return __float_as_uint(v);
    else if constexpr (TY == REPOPS_TYPE_F16) return __half_as_ushort(__float2half_rn(v));
    else return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Two half-precision values in a word, the first in the low half.
template <int TY>
__device__ __forceinline__ uint32_t narrowed2(float lo, float hi) {
    if constexpr (TY == REPOPS_TYPE_F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <int TY>
__device__ __forceinline__ void store_one(const DbgAccess &d, void *p, int64_t i, float v) {
    if constexpr (TY == REPOPS_TYPE_F32) store_global(d, static_cast<float *>(p) + i, v);
    else store_global(d, static_cast<uint16_t *>(p) + i, uint16_t(narrowed<TY>(v)));
}

// Elements i .. i+3, i a multiple of 4 elements from an aligned base.
template <int TY>
__device__ __forceinline__ float4 load_four(const DbgAccess &d, const void *p, int64_t i) {
    if constexpr (TY == REPOPS_TYPE_F32) {
        return load_once(d, reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
    } else {
        const uint2 w = load_once(d, reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i));
        if constexpr (TY == REPOPS_TYPE_BF16) {
            return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                               __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
        } else {
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
            return make_float4(a.x, a.y, b.x, b.y);
        }
    }
}

template <int TY>
__device__ __forceinline__ void store_four(const DbgAccess &d, void *p, int64_t i, float4 v) {
    if constexpr (TY == REPOPS_TYPE_F32) {
        store_once(d, reinterpret_cast<float4 *>(static_cast<float *>(p) + i), v);
    } else {
        store_once(d, reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i),
                   make_uint2(narrowed<TY>(v.x) | (narrowed<TY>(v.y) << 16), narrowed<TY>(v.z) | (narrowed<TY>(v.w) << 16)));
    }
}

}  // namespace
}  // namespace repops
