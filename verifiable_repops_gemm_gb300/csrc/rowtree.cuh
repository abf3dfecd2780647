// rowtree.cuh -- the fixed 32-ary reduction tree of the row operators and what
// the translation units that use it share: the swizzled shared-memory stage a
// row is held in, the tree over run results, one level of a column sum, and
// the host helpers that size their launches.
//
// A row's values are folded in runs of 32 (left to right from the first), the
// run results in runs of 32 again, level by level, until one value is left.
#pragma once

#include <algorithm>

#include "internal.cuh"

namespace repops {
namespace {

constexpr int RUN = 32;

__device__ __forceinline__ int64_t imin64(int64_t a, int64_t b) { return a < b ? a : b; }
constexpr int MAX_GENERIC_RUNS = 12288;         // run results in 48 KB of shared memory

// ------------------------------------------------------------ arithmetic ----

enum class Op { Sum, Max };

template <Op OP>
__device__ __forceinline__ float combine(float acc, float v) {
    if constexpr (OP == Op::Sum) return __fadd_rn(acc, v);
    else return v > acc ? v : acc;
}

// Upper levels of the tree over the m run results in a[] (shared memory),
// ping-ponging with b[]; every thread of the CTA calls it and receives the
// root.  Both buffers are clobbered.
template <Op OP>
__device__ float tree_upper(float *a, float *b, int m, float *bcast) {
    __syncthreads();
    while (m > 1) {
        const int groups = (m + RUN - 1) / RUN;
        for (int g = threadIdx.x; g < groups; g += blockDim.x) {
            const int s = g * RUN, e = min(s + RUN, m);
            float acc = a[s];
            for (int i = s + 1; i < e; ++i) acc = combine<OP>(acc, a[i]);
            b[g] = acc;
        }
        __syncthreads();
        float *t = a; a = b; b = t;
        m = groups;
    }
    if (threadIdx.x == 0) *bcast = a[0];
    __syncthreads();
    const float r = *bcast;
    __syncthreads();
    return r;
}

struct Square {
    __device__ __forceinline__ float operator()(float x) const { return __fmul_rn(x, x); }
};

// Run u of a row occupies 128 bytes of the stage at u*128; its 16-byte chunk c
// sits in slot c ^ (u & 7).  Eight consecutive lanes then hit eight different
// bank groups both when they copy eight consecutive chunks of one run and when
// each reads the same chunk of its own run.
__device__ __forceinline__ int stage_slot(int u, int c) { return u * 8 + (c ^ (u & 7)); }

// Tree reduction over i in [0, n) of f(i) (an index functor), as generic_reduce.
template <Op OP, class F>
__device__ float generic_reduce_idx(int64_t n, F f, float *buf, float *buf2, float *bcast) {
    const int runs = int((n + RUN - 1) / RUN);
    for (int j = threadIdx.x; j < runs; j += blockDim.x) {
        const int64_t s = int64_t(j) * RUN, e = imin64(s + RUN, n);
        float acc = f(s);
        for (int64_t i = s + 1; i < e; ++i) acc = combine<OP>(acc, f(i));
        buf[j] = acc;
    }
    return tree_upper<OP>(buf, buf2, runs, bcast);
}

// One tree level of a column sum: out[q][j] = fold of rows [32q, 32q + 32) of
// column j (left to right from the first).  Threads run along columns
// (coalesced), the grid's y dimension along q.
[[maybe_unused]] __global__ void __launch_bounds__(256)
colsum_pass_kernel(int64_t rows, int64_t cols, const float *__restrict__ x, int64_t ldx, float *__restrict__ out,
                   int64_t ldo, DbgAccess dbg) {
    const int64_t groups = (rows + RUN - 1) / RUN;
    for (int64_t q = blockIdx.y; q < groups; q += gridDim.y) {
        const int64_t r0 = q * RUN, r1 = imin64(r0 + RUN, rows);
        for (int64_t j = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; j < cols;
             j += int64_t(gridDim.x) * blockDim.x) {
            float acc = load_global(dbg, x + r0 * ldx + j);
            for (int64_t i = r0 + 1; i < r1; ++i) acc = __fadd_rn(acc, load_global(dbg, x + i * ldx + j));
            store_global(dbg, out + q * ldo + j, acc);
        }
    }
}

// ------------------------------------------------------------ host ----

[[maybe_unused]] int grid_for_rows(int64_t rows) {
    DeviceInfo di;
    const int sms = current_device_info(&di) == REPOPS_OK ? di.sms : 152;
    return int(std::min<int64_t>(rows, int64_t(sms) * 32));
}

// Launches `kern` with as many CTAs as fit on the device at once (at most one
// per row); each CTA then strides over the rows.
template <class Kern, class... Args>
int launch_persistent(Kern kern, int threads, size_t smem, int64_t rows, cudaStream_t s, Args... args) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return set_cuda_error(e);
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
    if (e != cudaSuccess) return set_cuda_error(e);
    DeviceInfo di;
    const int sms = current_device_info(&di) == REPOPS_OK ? di.sms : 152;
    const int grid = int(std::min<int64_t>(rows, int64_t(std::max(per_sm, 1)) * sms));
    kern<<<grid, threads, smem, s>>>(args...);
    return check_launch();
}

// Span check for a rows x cols operand with pitch ld; false on overflow.
[[maybe_unused]] bool rows_span(int64_t rows, int64_t cols, int64_t ld, uint64_t *bytes) {
    if (rows == 0 || cols == 0) { *bytes = 0; return true; }
    if (ld < cols || rows - 1 > (INT64_MAX / 4 - cols) / ld) return false;
    *bytes = uint64_t((rows - 1) * ld + cols) * 4u;
    return true;
}

}  // namespace
}  // namespace repops
