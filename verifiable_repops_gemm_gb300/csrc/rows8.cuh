// rows8.cuh -- the 8-bit row format: whole numbers q in [-127, 127] with one
// binary32 scale for every `group` consecutive columns of a row (group 0: one
// for the whole row); q stands for fl(q * scale).  Shared by the kernels that
// write it and those that read it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.cuh"

namespace repops {
namespace {

// column >> shift is the column's group; group 0 puts every column in group 0
// (columns are below 2^31)
inline int group_shift(int64_t group) {
    int s = 0;
    if (group == 0) return 31;
    while ((int64_t(1) << s) < group) ++s;
    return s;
}

// Groups are whole runs of the 32-ary tree, so that a run has one scale.
inline bool known_group(int64_t group) {
    return group == 0 || group == 32 || group == 64 || group == 128 || group == 256;
}

inline int64_t group_count(int64_t cols, int64_t group) { return group == 0 ? 1 : (cols + group - 1) / group; }

[[maybe_unused]] inline bool known_storage(int t) {
    return t == REPOPS_TYPE_F32 || t == REPOPS_TYPE_F16 || t == REPOPS_TYPE_BF16;
}
[[maybe_unused]] inline unsigned storage_size(int t) { return t == REPOPS_TYPE_F32 ? 4u : 2u; }

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

// Four whole numbers packed in a word, lowest byte first, each as the value it
// stands for: one rounding, fl(q * scale).  With its sign bit flipped a byte is
// q + 128; as the low byte of 2^23's pattern it is 2^23 + q + 128, and taking
// 2^23 + 128 away is exact -- a permute and an add, where the conversion
// instruction runs at an eighth of their rate.
__device__ __forceinline__ float4 unpack_q4(uint32_t w, float scale) {
    const uint32_t u = w ^ 0x80808080u;
    const float a = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540)), b = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7541)),
                c = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7542)), d = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7543));
    return make_float4(__fmul_rn(__fsub_rn(a, 8388736.0f), scale), __fmul_rn(__fsub_rn(b, 8388736.0f), scale),
                       __fmul_rn(__fsub_rn(c, 8388736.0f), scale), __fmul_rn(__fsub_rn(d, 8388736.0f), scale));
}

// One of them.
__device__ __forceinline__ float unpack_q1(int8_t q, float scale) {
    const uint32_t u = 0x4b000000u | (uint32_t(uint8_t(q)) ^ 0x80u);
    return __fmul_rn(__fsub_rn(__uint_as_float(u), 8388736.0f), scale);
}

}  // namespace
}  // namespace repops
