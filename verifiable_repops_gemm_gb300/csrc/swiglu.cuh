// swiglu.cuh -- the arithmetic of the SiLU-gated MLP activation and its
// backward, and the overlap checks of column blocks, shared by the kernels that
// read binary32 activations and those that read 8-bit ones.
#pragma once

#include "fixed_math.cuh"
#include "internal.cuh"

namespace repops {
namespace {

__device__ __forceinline__ float sigmoid_fixed(float x) {
    return __frcp_rn(__fadd_rn(1.0f, exp_fixed(-x)));   // correctly rounded 1/(1 + e)
}

// Two sigmoids: the same steps lane by lane, the exponentials and the 1 + e
// additions of the pair as packed adds (exp_fixed2): the same bits.
__device__ __forceinline__ float2 sigmoid_fixed2(float x0, float x1) {
    const float2 e = exp_fixed2(-x0, -x1);
    float d0, d1;
    unpack2(add2_rn(pack2(1.0f, 1.0f), pack2(e.x, e.y)), d0, d1);
    return make_float2(__frcp_rn(d0), __frcp_rn(d1));
}

__device__ __forceinline__ float swiglu1(float g, float u) {
    return __fmul_rn(__fmul_rn(g, sigmoid_fixed(g)), u);
}

__device__ __forceinline__ float swiglu_s(float g, float u, float sg) {
    return __fmul_rn(__fmul_rn(g, sg), u);
}

__device__ __forceinline__ void swiglu_grad_s(float g, float u, float dh, float sg, float &dg, float &du) {
    du = __fmul_rn(dh, __fmul_rn(g, sg));
    const float t = __fmul_rn(dh, u);
    const float d = __fmul_rn(sg, __fadd_rn(1.0f, __fmul_rn(g, __fsub_rn(1.0f, sg))));
    dg = __fmul_rn(t, d);
}

__device__ __forceinline__ void swiglu_grad1(float g, float u, float dh, float &dg, float &du) {
    swiglu_grad_s(g, u, dh, sigmoid_fixed(g), dg, du);
}

// ------------------------------------------------------------------- host ----

[[maybe_unused]] bool span2d(int64_t rows, int64_t cols, int64_t ld, uint64_t *bytes) {
    if (rows == 0 || cols == 0) { *bytes = 0; return true; }
    if (ld < cols || rows - 1 > (INT64_MAX / 4 - cols) / ld) return false;
    *bytes = uint64_t((rows - 1) * ld + cols) * 4u;
    return true;
}

// True when two rows x cols blocks of floats, at a (pitch lda) and b (pitch
// ldb), share an element.  With one pitch the test is exact, so column
// blocks of one matrix ([g | u] side by side) do not count as overlapping;
// with two pitches it falls back to the byte spans.
bool blocks_overlap(const float *a, int64_t lda, const float *b, int64_t ldb, int64_t rows, int64_t cols) {
    uint64_t ab = 0, bb = 0;
    span2d(rows, cols, lda, &ab);
    span2d(rows, cols, ldb, &bb);
    if (!ranges_overlap(a, ab, b, bb)) return false;
    const intptr_t db = reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a);
    if (lda != ldb || db % 4 != 0) return true;
    // b = a + d elements: b's row r starts in a's row r + q at column rem
    const int64_t d = db / 4;
    int64_t q = d / lda, rem = d % lda;
    if (rem < 0) { rem += lda; --q; }
    auto rows_meet = [&](int64_t shift) { return shift > -rows && shift < rows; };
    if (rem < cols && rows_meet(q)) return true;               // columns [rem, rem + cols) of row r + q
    if (rem + cols > lda && rows_meet(q + 1)) return true;     // the part wrapping into row r + q + 1
    return false;
}

// `out` may be `in` itself with the same pitch; any other shared element is
// an alias.
[[maybe_unused]] bool bad_overlap(const float *out, int64_t ldo, const float *in, int64_t ldi, int64_t rows, int64_t cols) {
    if (out == in && ldo == ldi) return false;
    return blocks_overlap(out, ldo, in, ldi, rows, cols);
}

}  // namespace
}  // namespace repops
