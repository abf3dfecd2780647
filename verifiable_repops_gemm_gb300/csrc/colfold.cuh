// colfold.cuh -- the last levels of a column sum whose run results (32 rows each,
// see rowtree.cuh) a kernel has left in scratch, and that scratch.
#pragma once

#include "rowtree.cuh"

namespace repops {
namespace {

[[maybe_unused]] inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t MAX_FOLD_ROWS = RUN * RUN;    // run results the last fold takes

struct FoldSet {
    const float *in;        // blocks x runs x n run results
    float *out;             // blocks x n, pitch ldo
    int64_t blocks, runs, ldo;
};
struct FoldArgs : DbgAccess {
    FoldSet s[3];
    int64_t n;
};

// The two levels of the tree over up to 1024 run results: 32 columns a CTA, a
// warp for each run of 32 results (as many as the longest sum has).
[[maybe_unused]] __global__ void __launch_bounds__(1024) column_fold_kernel(FoldArgs a) {
    __shared__ float part[RUN][RUN + 1];
    const FoldSet s = a.s[blockIdx.z];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = blockIdx.x * int64_t(RUN) + tx;
    const int groups = int((s.runs + RUN - 1) / RUN);
    grid_wait();
    for (int64_t b = blockIdx.y; b < s.blocks; b += gridDim.y) {
        const int64_t r0 = int64_t(ty) * RUN, r1 = imin64(r0 + RUN, s.runs);
        if (c < a.n && r0 < r1) {
            const float *in = s.in + (b * s.runs + r0) * a.n + c;
            float acc = load_global(a, in);
            const int m = int(r1 - r0);
            if (m == RUN) {
#pragma unroll
                for (int i = 1; i < RUN; ++i) acc = __fadd_rn(acc, load_global(a, in + int64_t(i) * a.n));
            } else {
                for (int i = 1; i < m; ++i) acc = __fadd_rn(acc, load_global(a, in + int64_t(i) * a.n));
            }
            part[ty][tx] = acc;
        }
        __syncthreads();
        if (ty == 0 && c < a.n) {
            float acc = part[0][tx];
            for (int g = 1; g < groups; ++g) acc = __fadd_rn(acc, part[g][tx]);
            store_global(a, s.out + b * s.ldo + c, acc);
        }
        __syncthreads();
    }
}

// Device scratch of a call: the caller's, or the library's pool's.
struct Workspace {
    float *p = nullptr;
    bool pool = false;
    cudaStream_t stream;
    int get(void *ws, uint64_t ws_bytes, uint64_t need, cudaStream_t s) {
        stream = s;
        if (ws) {
            if (ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 16 != 0) return REPOPS_ERR_INVALID_ARG;
            p = static_cast<float *>(ws);
            return REPOPS_OK;
        }
        if (scratch_malloc(reinterpret_cast<void **>(&p), size_t(need), s) != cudaSuccess) {
            cudaGetLastError();
            return REPOPS_ERR_ALLOC;
        }
        pool = true;
        return REPOPS_OK;
    }
    int release(int rc) {
        if (pool && p) {
            const cudaError_t e = cudaFreeAsync(p, stream);
            if (rc == REPOPS_OK && e != cudaSuccess) rc = set_cuda_error(e);
        }
        return rc;
    }
};

}  // namespace
}  // namespace repops
