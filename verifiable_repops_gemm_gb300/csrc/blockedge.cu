// blockedge.cu -- the edge between two blocks of a pre-norm transformer in one
// pass: the norm after a block, its gate and residual scale, the residual sum,
// and the norm before the next block; its backward pass; and RMSNorm's backward
// from an input kept in 8 bits.
//
//   p = RMSNorm(f; post),  y = x + alpha * (gate * p),  h = RMSNorm(y; pre)
//
// Every step is the one the separate operators take (rowops.cu): one binary32
// rounding each, row sums over the 32-ary tree, column sums over the tree of
// colsum, so the bits equal the separate operators' and only the memory
// traffic changes: forward 16 bytes an element (x, f in; y, h out) instead of
// 36, backward 24 (y, f, dy, dh in; dx, df out) plus what the column sums read.
//
// Row kernels: teams of T threads, a row a team at a time, a warp for each slab
// of 1024 columns.  The rows arrive by cp.async in a swizzled stage; element-wise
// steps take a slab in memory order (coalesced) and the tree takes it in run
// order, a run a lane, both from the stage.  Forward, a CTA is a team and reads
// the gains and the gate from the caches, with the next row's copies in flight
// (4096 x 2048: 29 us; a plain copy of as many bytes 23).  Backward, a row passes
// three dependent sums and takes about 6 us, so what counts is how many rows are
// in flight and how little each waits for: one CTA an SM holds as many teams as
// fit its shared memory and, once for all of them, the gains and the gate (read
// from the caches they were a third of a row's time: 8192 x 2048, 84 -> 67 us; a
// plain copy of as many bytes 60).
//
// Column sums (the gradients of the gains and the gate) need their terms
// folded in row order, a run of 32 rows at a time: a second kernel, a thread
// for each column (four with 16-byte rows) and run, forms the terms again from
// the rows and the row's 1/rms that the row kernel left, and a last one folds
// the run results.  Writing the terms and summing them afterwards would move 8
// bytes an element for each of the three sums instead of 16 for all.  8192 x
// 2048: 45 us for the terms, 4 for the last fold, 116 for the whole backward;
// taking the rows in pieces that stay in L2 lost more to the launches' ends
// than it saved (145 us in pieces of 2600 rows).
#include <algorithm>
#include <atomic>

#include "internal.cuh"
#include "rows8.cuh"
#include "rowtree.cuh"

namespace repops {
namespace {

constexpr int64_t MAX_STAGED_COLS = 8192;       // 256 threads, a run each
constexpr int64_t MAX_FOLD_ROWS = RUN * RUN;    // run results the last fold takes

// ------------------------------------------------------------- row slabs ----
// A warp's slab: step k (of KS, 8 but for short rows) covers four values a lane.  With 16-byte rows
// (VEC) they are columns 128k + 4*lane .. + 3 of the slab; else columns
// 128k + lane + {0, 32, 64, 96}.  `slab` is the slab's first column.

template <bool VEC>
__device__ __forceinline__ int slab_col(int slab, int k, int t) {
    const int lane = threadIdx.x & 31;
    return VEC ? slab + 128 * k + 4 * lane + t : slab + 128 * k + 32 * t + lane;
}

// Loads take no branch, so that a slab's are all in flight together: a column
// past the row's end reads column 0 instead, and its result is never stored or
// folded.  n is a multiple of 4 with VEC.
template <bool VEC>
__device__ __forceinline__ float4 row_load(const DbgAccess &d, const float *__restrict__ row, int slab, int k, int n) {
    const int c = slab_col<VEC>(slab, k, 0);
    if constexpr (VEC) {
        return load_const(d, reinterpret_cast<const float4 *>(row + (c < n ? c : 0)));
    } else {
        return make_float4(load_const(d, row + (c < n ? c : 0)), load_const(d, row + (c + 32 < n ? c + 32 : 0)),
                           load_const(d, row + (c + 64 < n ? c + 64 : 0)), load_const(d, row + (c + 96 < n ? c + 96 : 0)));
    }
}

// Asks for the warp's slab of a parameter row (may be null) ahead of its use.
__device__ __forceinline__ void row_prefetch(const float *row, int slab, int n) {
    if (!row) return;
    const int c = slab + 32 * (threadIdx.x & 31);              // a 128-byte line a lane
    if (c < n) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + c));
}

// KEEP: the row is read again soon (by the column sums); else its lines make
// way first.
template <bool VEC, bool KEEP = true>
__device__ __forceinline__ void row_store(const DbgAccess &d, float *row, int slab, int k, int n, float4 v) {
    const int c = slab_col<VEC>(slab, k, 0);
    if constexpr (VEC) {
        if constexpr (KEEP) {
            if (c < n) store_global(d, reinterpret_cast<float4 *>(row + c), v);
        } else {
            if (c < n) store_once(d, reinterpret_cast<float4 *>(row + c), v);
        }
    } else {
        if (c < n) store_global(d, row + c, v.x);
        if (c + 32 < n) store_global(d, row + c + 32, v.y);
        if (c + 64 < n) store_global(d, row + c + 64, v.z);
        if (c + 96 < n) store_global(d, row + c + 96, v.w);
    }
}

// A slab step's place in the stage.
template <bool VEC>
__device__ __forceinline__ int stage_float(int slab, int k, int t) {
    const int lane = threadIdx.x & 31, u0 = slab / RUN + 4 * k;
    if constexpr (VEC) return 4 * stage_slot(u0 + (lane >> 3), lane & 7) + t;
    else return 4 * stage_slot(u0 + t, lane >> 2) + (lane & 3);
}

template <bool VEC>
__device__ __forceinline__ float4 stage_load(const float4 *stage, int slab, int k) {
    const float *s = reinterpret_cast<const float *>(stage);
    if constexpr (VEC) return *reinterpret_cast<const float4 *>(s + stage_float<VEC>(slab, k, 0));
    else
        return make_float4(s[stage_float<VEC>(slab, k, 0)], s[stage_float<VEC>(slab, k, 1)],
                           s[stage_float<VEC>(slab, k, 2)], s[stage_float<VEC>(slab, k, 3)]);
}

template <bool VEC>
__device__ __forceinline__ void stage_store(float4 *stage, int slab, int k, float4 v) {
    float *s = reinterpret_cast<float *>(stage);
    if constexpr (VEC) {
        *reinterpret_cast<float4 *>(s + stage_float<VEC>(slab, k, 0)) = v;
    } else {
        s[stage_float<VEC>(slab, k, 0)] = v.x;
        s[stage_float<VEC>(slab, k, 1)] = v.y;
        s[stage_float<VEC>(slab, k, 2)] = v.z;
        s[stage_float<VEC>(slab, k, 3)] = v.w;
    }
}

// Starts the copy of the warp's slab of a row into the stage.
template <bool VEC, int KS>
__device__ __forceinline__ void stage_row(const DbgAccess &d, float4 *stage, const float *row, int slab, int n) {
    float *s = reinterpret_cast<float *>(stage);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
        if constexpr (VEC) {
            const int c = slab_col<VEC>(slab, k, 0);
            if (c < n && REPOPS_DBG_READ(d, row + c, 16)) cp_async_16(s + stage_float<VEC>(slab, k, 0), row + c, 16u);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int c = slab_col<VEC>(slab, k, t);
                if (c < n && REPOPS_DBG_READ(d, row + c, 4)) cp_async_4(s + stage_float<VEC>(slab, k, t), row + c, 4u);
            }
        }
    }
}

// The CTA's copy of a parameter row (null: none), in memory order, and a slab
// step of it.  A barrier follows the copies.
template <int LEN>
__device__ __forceinline__ void param_copy(const DbgAccess &d, float *dst, const float *src, int n) {
    if (!src) return;
    for (int c = threadIdx.x; c < LEN; c += blockDim.x) dst[c] = c < n ? load_const(d, src + c) : 0.0f;
}

template <bool VEC>
__device__ __forceinline__ float4 param_load(const float *param, int slab, int k) {
    const int c = slab_col<VEC>(slab, k, 0);
    if constexpr (VEC) return *reinterpret_cast<const float4 *>(param + c);
    else return make_float4(param[c], param[c + 32], param[c + 64], param[c + 96]);
}

// The warp's group result of the tree over the staged values f(v): each lane
// folds its run, every lane folds the lanes' results in order.  `lanes`: 32
// floats of the warp's own.
template <class F>
__device__ __forceinline__ float slab_fold(const float4 *stage, float4 *lanes, int slab, int n, F f) {
    const int lane = threadIdx.x & 31, u = slab / RUN + lane;
    const int len = min(RUN, n - u * RUN);                 // 0 or less past the end
    const int at = len > 0 ? u : slab / RUN;               // a lane without a run reads one that is there
    float v[RUN];
#pragma unroll
    for (int c = 0; c < RUN / 4; ++c) {
        const float4 w = stage[stage_slot(at, c)];
        v[4 * c] = w.x; v[4 * c + 1] = w.y; v[4 * c + 2] = w.z; v[4 * c + 3] = w.w;
    }
    float acc = f(v[0]);
    if (len == RUN) {
#pragma unroll
        for (int i = 1; i < RUN; ++i) acc = __fadd_rn(acc, f(v[i]));
    } else {
#pragma unroll
        for (int i = 1; i < RUN; ++i)
            if (i < len) acc = __fadd_rn(acc, f(v[i]));
    }
    const int have = (n + RUN - 1) / RUN - slab / RUN;     // runs present from this warp on
    // the lanes' results to every lane: a store and eight broadcast reads (31
    // shuffles cost the shared-memory pipe three times as much)
    __syncwarp();
    reinterpret_cast<float *>(lanes)[lane] = acc;
    __syncwarp();
    float r[RUN];
#pragma unroll
    for (int c = 0; c < RUN / 4; ++c) {
        const float4 w = lanes[c];
        r[4 * c] = w.x; r[4 * c + 1] = w.y; r[4 * c + 2] = w.z; r[4 * c + 3] = w.w;
    }
    float g = r[0];
    if (have >= RUN) {
#pragma unroll
        for (int i = 1; i < RUN; ++i) g = __fadd_rn(g, r[i]);
    } else {
#pragma unroll
        for (int i = 1; i < RUN; ++i)
            if (i < have) g = __fadd_rn(g, r[i]);
    }
    return g;
}

// The tree's roots from the warps' group results (one barrier of the team).
// buf has two halves used in turn, so that a thread still reading one
// reduction's half never races the next one's writes.
template <int T, int NV>
__device__ __forceinline__ void slab_roots(float (&v)[NV], float (&buf)[2][2][8], int &phase, int team, int n) {
    if constexpr (T > 32) {
        const int warp = (threadIdx.x % T) >> 5;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int j = 0; j < NV; ++j) buf[phase][j][warp] = v[j];
        }
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(T) : "memory");
        const int G = (n + 1023) / 1024;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            v[j] = buf[phase][j][0];
            for (int k = 1; k < G; ++k) v[j] = __fadd_rn(v[j], buf[phase][j][k]);
        }
        phase ^= 1;
    }
}

__device__ __forceinline__ float rms_inv(float sum, float nf, float eps) {
    return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sum, nf), eps)));
}

__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
    return make_float4(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y), __fmul_rn(a.z, b.z), __fmul_rn(a.w, b.w));
}
__device__ __forceinline__ float4 mul4(float4 a, float s) { return mul4(a, make_float4(s, s, s, s)); }
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
}
__device__ __forceinline__ float4 sub4(float4 a, float4 b) {
    return make_float4(__fsub_rn(a.x, b.x), __fsub_rn(a.y, b.y), __fsub_rn(a.z, b.z), __fsub_rn(a.w, b.w));
}

struct Ident {
    __device__ __forceinline__ float operator()(float x) const { return x; }
};

// Teams of a CTA whose rows take STAGES stages and whose parameters PARAMS: what
// 224 KB hold, and 15 barriers at most.
template <int T, int KS, int STAGES, int PARAMS, int MAX_THREADS>
constexpr int kTeams = std::min({(224 * 1024 / (T * KS * 16) - PARAMS) / STAGES, MAX_THREADS / T, T > 32 ? 15 : 64});
template <int T, int KS, int STAGES, int PARAMS, int TEAMS>
constexpr size_t kTeamSmem = size_t(T) * KS * 16 * (PARAMS + STAGES * TEAMS);

// --------------------------------------------------------------- forward ----

struct EdgeArgs : DbgAccess {
    int64_t rows, n;
    const float *x, *f;
    int64_t ldx, ldf;
    const float *post, *gate, *pre;    // each may be null
    int64_t ldgate, gate_rows;
    float alpha, eps;
    float *y, *h;
    int64_t ldy, ldh;
};

// Two stages of rows where they leave room for a few CTAs.
template <int T>
constexpr bool kEdgePrefetch = T <= 128;

template <int T, int KS, bool VEC>
__global__ void __launch_bounds__(T, 512 / T) edge_forward_kernel(EdgeArgs p) {
    extern __shared__ float4 stage_mem[];
    __shared__ float roots[2][2][8];
    __shared__ float4 lane_mem[T / 4];
    if (!REPOPS_DBG_SMEM_OK(size_t(T) * KS * 16 * (kEdgePrefetch<T> ? 4 : 2), p.status)) return;
    float4 *lanes = lane_mem + (threadIdx.x >> 5) * 8;
    const int slab = (threadIdx.x >> 5) * 1024;
    int phase = 0;
    constexpr int Q = T * KS, KB = KS < 4 ? KS : 4;            // a stage in 16-byte chunks
    constexpr bool PF = kEdgePrefetch<T>;
    const int n = int(p.n);
    const float nf = float(p.n);
    int cur = 0;
    int64_t row = blockIdx.x;
    if (row < p.rows) {
        stage_row<VEC, KS>(p, stage_mem, p.f + row * p.ldf, slab, n);
        stage_row<VEC, KS>(p, stage_mem + Q, p.x + row * p.ldx, slab, n);
    }
    cp_async_commit();
    for (; row < p.rows; row += gridDim.x) {
        const int64_t next = row + gridDim.x;
        float4 *sf = stage_mem + cur * 2 * Q, *sx = sf + Q;
        if constexpr (PF) {
            cur ^= 1;
            if (next < p.rows) {
                stage_row<VEC, KS>(p, stage_mem + cur * 2 * Q, p.f + next * p.ldf, slab, n);
                stage_row<VEC, KS>(p, stage_mem + cur * 2 * Q + Q, p.x + next * p.ldx, slab, n);
            }
            cp_async_commit();
        }
        const float *gate = p.gate ? p.gate + (row / p.gate_rows) * p.ldgate : nullptr;
        if (row == blockIdx.x) {            // the parameters are on their way while the first row is
            row_prefetch(p.post, slab, n);
            row_prefetch(gate, slab, n);
            row_prefetch(p.pre, slab, n);
        }
        cp_async_wait<PF ? 1 : 0>();
        __syncwarp();
        float inv_f = 0.0f;
        if (p.post) {
            float s[1] = {slab_fold(sf, lanes, slab, n, Square())};
            slab_roots<T, 1>(s, roots, phase, 0, n);
            inv_f = rms_inv(s[0], nf, p.eps);
        }
        float *yr = p.y + row * p.ldy;
#pragma unroll
        for (int b = 0; b < KS; b += KB) {    // up to four steps' loads in flight together
            float4 w[KB], g[KB];
            if (p.post) {
#pragma unroll
                for (int k = 0; k < KB; ++k) w[k] = row_load<VEC>(p, p.post, slab, b + k, n);
            }
            if (gate) {
#pragma unroll
                for (int k = 0; k < KB; ++k) g[k] = row_load<VEC>(p, gate, slab, b + k, n);
            }
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                float4 v = stage_load<VEC>(sf, slab, b + k);
                if (p.post) v = mul4(mul4(v, inv_f), w[k]);
                if (gate) v = mul4(v, g[k]);
                v = add4(stage_load<VEC>(sx, slab, b + k), mul4(v, p.alpha));
                row_store<VEC>(p, yr, slab, b + k, n, v);
                if (p.pre) stage_store<VEC>(sx, slab, b + k, v);
            }
        }
        if (p.pre) {
            __syncwarp();
            float s[1] = {slab_fold(sx, lanes, slab, n, Square())};
            slab_roots<T, 1>(s, roots, phase, 0, n);
            const float inv_y = rms_inv(s[0], nf, p.eps);
            float *hr = p.h + row * p.ldh;
            float4 w[KS];
#pragma unroll
            for (int k = 0; k < KS; ++k) w[k] = row_load<VEC>(p, p.pre, slab, k, n);
#pragma unroll
            for (int k = 0; k < KS; ++k) row_store<VEC>(p, hr, slab, k, n, mul4(mul4(stage_load<VEC>(sx, slab, k), inv_y), w[k]));
        }
        __syncwarp();                       // the stage is read before it is filled again
        if constexpr (!PF) {
            if (next < p.rows) {
                stage_row<VEC, KS>(p, sf, p.f + next * p.ldf, slab, n);
                stage_row<VEC, KS>(p, sx, p.x + next * p.ldx, slab, n);
            }
            cp_async_commit();
        }
    }
    cp_async_wait<0>();
}

// Rows of more than 8192 values: each phase reads the row again.
__global__ void __launch_bounds__(256) edge_forward_long_kernel(EdgeArgs p) {
    extern __shared__ float buf[];
    __shared__ float bcast;
    const int runs = int((p.n + RUN - 1) / RUN);
    if (!REPOPS_DBG_SMEM_OK(uint64_t(runs + (runs + RUN - 1) / RUN) * sizeof(float), p.status)) return;
    float *buf2 = buf + runs;
    const float nf = float(p.n);
    auto at = [&](const float *v) { return load_global(p, v); };
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float *xr = p.x + row * p.ldx, *fr = p.f + row * p.ldf;
        const float *gate = p.gate ? p.gate + (row / p.gate_rows) * p.ldgate : nullptr;
        float *yr = p.y + row * p.ldy;
        float inv_f = 0.0f;
        if (p.post)
            inv_f = rms_inv(generic_reduce_idx<Op::Sum>(
                                p.n, [&](int64_t i) { const float v = at(fr + i); return __fmul_rn(v, v); }, buf, buf2,
                                &bcast),
                            nf, p.eps);
        for (int64_t i = threadIdx.x; i < p.n; i += 256) {
            float v = at(fr + i);
            if (p.post) v = __fmul_rn(__fmul_rn(v, inv_f), at(p.post + i));
            if (gate) v = __fmul_rn(v, at(gate + i));
            store_global(p, yr + i, __fadd_rn(at(xr + i), __fmul_rn(p.alpha, v)));
        }
        __syncthreads();
        if (p.pre) {
            const float inv_y = rms_inv(generic_reduce_idx<Op::Sum>(
                                            p.n, [&](int64_t i) { const float v = at(yr + i); return __fmul_rn(v, v); }, buf,
                                            buf2, &bcast),
                                        nf, p.eps);
            float *hr = p.h + row * p.ldh;
            for (int64_t i = threadIdx.x; i < p.n; i += 256) 
                store_global(p, hr + i, __fmul_rn(__fmul_rn(at(yr + i), inv_y), at(p.pre + i)));
        }
        __syncthreads();
    }
}

// -------------------------------------------------------------- backward ----

struct EdgeBackArgs : DbgAccess {
    int64_t rows, n;
    // the norm before the next block: its input y (or q, s: 8 bits), the
    // gradient dh of its output, and the gradient dy arriving past it
    const float *y;
    int64_t ldy;
    const int8_t *q;
    int64_t ldq;
    const float *s;
    int64_t lds;
    int shift;
    const float *dh, *dy;              // either may be null
    int64_t lddh, lddy;
    const float *pre;
    // the block's output, its norm and gate (only with F)
    const float *f;
    int64_t ldf;
    const float *post, *gate;          // each may be null
    int64_t ldgate, gate_rows;
    float alpha, eps;
    float *dx, *df, *h;                // h: the norm's output again, only from 8 bits
    int64_t lddx, lddf, ldh;
    float *inv_y, *inv_f;              // a row's 1/rms, for the column sums
};

template <bool VEC>
__device__ __forceinline__ float4 row8_load(const EdgeBackArgs &p, int64_t row, int slab, int k, int n) {
    const int c = slab_col<VEC>(slab, k, 0);
    const int8_t *q = p.q + row * p.ldq;
    const float *s = p.s + row * p.lds;
    if constexpr (VEC) {                   // a group is a multiple of 4 columns
        const int i = c < n ? c : 0;
        return unpack_q4(load_const(p, reinterpret_cast<const uint32_t *>(q + i)), load_const(p, s + (i >> p.shift)));
    } else {
        float v[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int i = c + 32 * t < n ? c + 32 * t : 0;
            v[t] = unpack_q1(load_const(p, q + i), load_const(p, s + (i >> p.shift)));
        }
        return make_float4(v[0], v[1], v[2], v[3]);
    }
}

// Stages of a row: y, dh, dy, and f with F; parameters: pre, and post and the
// gate with F (whose rows want 160 registers a thread).
template <int T, int KS, bool F>
constexpr int kBackTeams = F ? kTeams<T, KS, 4, 3, KS == 8 ? 384 : 512> : kTeams<T, KS, 3, 1, 512>;

// dx = RMSNorm'(y; dh) + dy, then, with F, df through the gate and the norm
// after the block.  Q8: y comes in 8 bits, and h may be written again.
template <int T, int KS, bool VEC, bool Q8, bool F>
__global__ void __launch_bounds__(T *kBackTeams<T, KS, F>, 1) edge_backward_kernel(EdgeBackArgs p) {
    constexpr int Q = T * KS, TEAMS = kBackTeams<T, KS, F>;
    extern __shared__ float4 smem[];
    __shared__ float roots[TEAMS][2][2][8];
    __shared__ float4 lane_mem[TEAMS * T / 4];
    if (!REPOPS_DBG_SMEM_OK((F ? kTeamSmem<T, KS, 4, 3, TEAMS> : kTeamSmem<T, KS, 3, 1, TEAMS>), p.status)) return;
    const int n = int(p.n), team = threadIdx.x / T, slab = ((threadIdx.x % T) >> 5) * 1024;
    const float nf = float(p.n);
    float *pre = reinterpret_cast<float *>(smem), *post = pre + 4 * Q, *gate1 = post + 4 * Q;
    float4 *sy = smem + (F ? 3 : 1) * Q + team * Q * (F ? 4 : 3), *sh = sy + Q, *sr = sh + Q, *sf = sr + Q;
    float4 *lanes = lane_mem + (threadIdx.x >> 5) * 8;
    const bool one_gate = F && p.gate && p.gate_rows >= p.rows;
    param_copy<4 * Q>(p, pre, p.pre, n);
    if constexpr (F) {
        param_copy<4 * Q>(p, post, p.post, n);
        param_copy<4 * Q>(p, gate1, one_gate ? p.gate : nullptr, n);
    }
    __syncthreads();
    int phase = 0;
    // rows go to the SMs first, then to their teams
    for (int64_t row = int64_t(team) * gridDim.x + blockIdx.x; row < p.rows; row += int64_t(gridDim.x) * TEAMS) {
        if (p.dh) {
            if constexpr (!Q8) stage_row<VEC, KS>(p, sy, p.y + row * p.ldy, slab, n);
            stage_row<VEC, KS>(p, sh, p.dh + row * p.lddh, slab, n);
        }
        if constexpr (F) stage_row<VEC, KS>(p, sf, p.f + row * p.ldf, slab, n);
        cp_async_commit();
        if (p.dy) stage_row<VEC, KS>(p, sr, p.dy + row * p.lddy, slab, n);
        cp_async_commit();
        if constexpr (Q8) {
#pragma unroll
            for (int k = 0; k < KS; ++k) stage_store<VEC>(sy, slab, k, row8_load<VEC>(p, row, slab, k, n));
        }
        cp_async_wait<1>();
        __syncwarp();
        float r2[2] = {0.0f, 0.0f};
        if (p.dh) r2[0] = slab_fold(sy, lanes, slab, n, Square());
        if constexpr (F) {
            if (p.post) r2[1] = slab_fold(sf, lanes, slab, n, Square());
        }
        slab_roots<T, 2>(r2, roots[team], phase, team, n);
        const float inv_y = rms_inv(r2[0], nf, p.eps), inv_f = rms_inv(r2[1], nf, p.eps);
        if (threadIdx.x % T == 0) {
            if (p.dh) store_global(p, p.inv_y + row, inv_y);
            if constexpr (F) {
                if (p.post) store_global(p, p.inv_f + row, inv_f);
            }
        }
        float4 e[KS];                             // dx
        if (p.dh) {
            // sh <- gy * xh, summed from there
            float4 g[KS];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                g[k] = param_load<VEC>(pre, slab, k);
                e[k] = mul4(stage_load<VEC>(sy, slab, k), inv_y);
                if constexpr (Q8) {
                    if (p.h) row_store<VEC, false>(p, p.h + row * p.ldh, slab, k, n, mul4(e[k], g[k]));
                }
                g[k] = mul4(stage_load<VEC>(sh, slab, k), g[k]);
                stage_store<VEC>(sh, slab, k, mul4(g[k], e[k]));
            }
            __syncwarp();
            float r1[1] = {slab_fold(sh, lanes, slab, n, Ident())};
            slab_roots<T, 1>(r1, roots[team], phase, team, n);
            const float c = __fdiv_rn(r1[0], nf);
#pragma unroll
            for (int k = 0; k < KS; ++k) e[k] = mul4(sub4(g[k], mul4(e[k], c)), inv_y);
        }
        cp_async_wait<0>();
        __syncwarp();
        if (p.dy) {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const float4 d = stage_load<VEC>(sr, slab, k);
                e[k] = p.dh ? add4(e[k], d) : d;
            }
        }
        float *dxr = p.dx + row * p.lddx;
#pragma unroll
        for (int k = 0; k < KS; ++k) row_store<VEC>(p, dxr, slab, k, n, e[k]);
        if constexpr (F) {
            float *dfr = p.df + row * p.lddf;
            const float *gate = p.gate && !one_gate ? p.gate + (row / p.gate_rows) * p.ldgate : nullptr;
            float4 g[KS];
            if (gate) {
#pragma unroll
                for (int k = 0; k < KS; ++k) g[k] = row_load<VEC>(p, gate, slab, k, n);
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                e[k] = mul4(e[k], p.alpha);
                if (gate) e[k] = mul4(e[k], g[k]);
                else if (one_gate) e[k] = mul4(e[k], param_load<VEC>(gate1, slab, k));
            }
            if (p.post) {
                __syncwarp();
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    e[k] = mul4(e[k], param_load<VEC>(post, slab, k));
                    g[k] = mul4(stage_load<VEC>(sf, slab, k), inv_f);
                    stage_store<VEC>(sh, slab, k, mul4(e[k], g[k]));
                }
                __syncwarp();
                float r1[1] = {slab_fold(sh, lanes, slab, n, Ident())};
                slab_roots<T, 1>(r1, roots[team], phase, team, n);
                const float c = __fdiv_rn(r1[0], nf);
#pragma unroll
                for (int k = 0; k < KS; ++k) e[k] = mul4(sub4(e[k], mul4(g[k], c)), inv_f);
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) row_store<VEC, false>(p, dfr, slab, k, n, e[k]);
        }
        __syncwarp();
    }
    cp_async_wait<0>();
}

// Rows of more than 8192 values: each phase reads the row again.
template <bool Q8, bool F>
__global__ void __launch_bounds__(256) edge_backward_long_kernel(EdgeBackArgs p) {
    extern __shared__ float buf[];
    __shared__ float bcast;
    const int runs = int((p.n + RUN - 1) / RUN);
    if (!REPOPS_DBG_SMEM_OK(uint64_t(runs + (runs + RUN - 1) / RUN) * sizeof(float), p.status)) return;
    float *buf2 = buf + runs;
    const float nf = float(p.n);
    auto at = [&](const float *v) { return load_global(p, v); };
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        auto yv = [&](int64_t i) {
            if constexpr (Q8) return __fmul_rn(float(load_global(p, p.q + row * p.ldq + i)), at(p.s + row * p.lds + (i >> p.shift)));
            else return at(p.y + row * p.ldy + i);
        };
        const float *dhr = p.dh + row * p.lddh, *dyr = p.dy + row * p.lddy;
        float *dxr = p.dx + row * p.lddx;
        float inv_y = 0.0f, c = 0.0f;
        if (p.dh) {
            inv_y = rms_inv(generic_reduce_idx<Op::Sum>(
                                p.n, [&](int64_t i) { const float v = yv(i); return __fmul_rn(v, v); }, buf, buf2,
                                &bcast), nf, p.eps);
            c = __fdiv_rn(generic_reduce_idx<Op::Sum>(p.n, [&](int64_t i) {
                return __fmul_rn(__fmul_rn(at(dhr + i), at(p.pre + i)), __fmul_rn(yv(i), inv_y));
            }, buf, buf2, &bcast), nf);
            if (threadIdx.x == 0) store_global(p, p.inv_y + row, inv_y);
        }
        for (int64_t i = threadIdx.x; i < p.n; i += 256) {
            float d = 0.0f;
            if (p.dh) {
                const float xh = __fmul_rn(yv(i), inv_y);
                d = __fmul_rn(inv_y, __fsub_rn(__fmul_rn(at(dhr + i), at(p.pre + i)), __fmul_rn(xh, c)));
                if constexpr (Q8) {
                    if (p.h) store_global(p, p.h + row * p.ldh + i, __fmul_rn(xh, at(p.pre + i)));
                }
            }
            if (p.dy) d = p.dh ? __fadd_rn(d, at(dyr + i)) : at(dyr + i);
            store_global(p, dxr + i, d);
        }
        __syncthreads();
        if constexpr (F) {
            const float *fr = p.f + row * p.ldf;
            const float *gate = p.gate ? p.gate + (row / p.gate_rows) * p.ldgate : nullptr;
            float *dfr = p.df + row * p.lddf;
            auto dp = [&](int64_t i) {
                float d = __fmul_rn(at(dxr + i), p.alpha);
                if (gate) d = __fmul_rn(d, at(gate + i));
                return p.post ? __fmul_rn(d, at(p.post + i)) : d;
            };
            float inv_f = 0.0f, cf = 0.0f;
            if (p.post) {
                inv_f = rms_inv(generic_reduce_idx<Op::Sum>(
                                    p.n, [&](int64_t i) { const float v = at(fr + i); return __fmul_rn(v, v); }, buf, buf2,
                                    &bcast),
                                nf, p.eps);
                cf = __fdiv_rn(generic_reduce_idx<Op::Sum>(
                                   p.n, [&](int64_t i) { return __fmul_rn(dp(i), __fmul_rn(at(fr + i), inv_f)); }, buf, buf2,
                                   &bcast), nf);
                if (threadIdx.x == 0) store_global(p, p.inv_f + row, inv_f);
            }
            for (int64_t i = threadIdx.x; i < p.n; i += 256) {
                const float d = dp(i);
                store_global(p, dfr + i, p.post ? __fmul_rn(inv_f, __fsub_rn(d, __fmul_rn(__fmul_rn(at(fr + i), inv_f), cf))) : d);
            }
            __syncthreads();
        }
    }
}

// ------------------------------------------------------------ column sums ----

struct ColArgs {
    EdgeBackArgs e;
    int64_t block_rows;     // rows of a block: its runs of 32 start at its first row
    int64_t block_runs;     // runs of a block
    int64_t runs;           // runs in all
    float *pre, *post, *gate;   // run results, runs x n each; null: not wanted
    int64_t ldg;                // pitch of gate's (the others are packed)
};

template <int W>
struct Cols {
    float v[W];
};

template <int W>
__device__ __forceinline__ Cols<W> cols_load(const DbgAccess &d, const float *q) {
    Cols<W> r;
    if constexpr (W == 4) {
        const float4 w = load_const(d, reinterpret_cast<const float4 *>(q));
        r.v[0] = w.x; r.v[1] = w.y; r.v[2] = w.z; r.v[3] = w.w;
    } else {
        r.v[0] = load_const(d, q);
    }
    return r;
}

template <int W>
__device__ __forceinline__ void cols_store(const DbgAccess &d, float *q, const Cols<W> &r) {
    if constexpr (W == 4) store_global(d, reinterpret_cast<float4 *>(q), make_float4(r.v[0], r.v[1], r.v[2], r.v[3]));
    else store_global(d, q, r.v[0]);
}

// A thread forms and folds the terms of W columns over a run of 32 rows:
//   pre:  dh * (y * inv_y)
//   post: ((alpha * dx) * gate) * (f * inv_f)
//   gate: (alpha * dx) * ((f * inv_f) * post)
// PRE, POST, GATE: the sums wanted; eight rows' loads are in flight together.
template <int W, bool Q8, bool PRE, bool POST, bool GATE>
__global__ void __launch_bounds__(128) edge_columns_kernel(ColArgs a) {
    const EdgeBackArgs &p = a.e;
    constexpr int B = 8;                 // rows loaded at once; RUN is a multiple
    grid_release();
    const int64_t c = (blockIdx.x * int64_t(128) + threadIdx.x) * W;
    if (c >= p.n) return;
    Cols<W> post{};
    if (GATE && p.post) post = cols_load<W>(p, p.post + c);
    // the last rows first: the row kernel has just left them in L2
    for (int64_t run = a.runs - 1 - blockIdx.y; run >= 0; run -= gridDim.y) {
        const int64_t b = run / a.block_runs, first = b * a.block_rows + (run - b * a.block_runs) * RUN;
        const int rows = int(imin64(RUN, (b + 1) * a.block_rows - first));
        Cols<W> s_pre, s_post, s_gate, gate{};
        int64_t gate_left = 0;           // rows until the next gate row begins
        const float *gate_row = nullptr;
        if (POST && p.gate) {
            gate_row = p.gate + (first / p.gate_rows) * p.ldgate + c;
            gate_left = p.gate_rows - first % p.gate_rows;
            gate = cols_load<W>(p, gate_row);
        }
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += B) {
            Cols<W> y[B], d[B], dx[B], f[B];
            float iy[B], jf[B];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int64_t r = first + min(r0 + i, rows - 1);     // past the run: its last row, not folded
                if constexpr (PRE) {
                    if constexpr (Q8) {
                        const float s = load_const(p, p.s + r * p.lds + (c >> p.shift));
                        if constexpr (W == 4) {
                            const float4 w = unpack_q4(load_const(p, reinterpret_cast<const uint32_t *>(p.q + r * p.ldq + c)), s);
                            y[i].v[0] = w.x; y[i].v[1] = w.y; y[i].v[2] = w.z; y[i].v[3] = w.w;
                        } else {
                            y[i].v[0] = unpack_q1(load_const(p, p.q + r * p.ldq + c), s);
                        }
                    } else {
                        y[i] = cols_load<W>(p, p.y + r * p.ldy + c);
                    }
                    d[i] = cols_load<W>(p, p.dh + r * p.lddh + c);
                    iy[i] = load_const(p, p.inv_y + r);
                }
                if constexpr (POST || GATE) {
                    dx[i] = cols_load<W>(p, p.dx + r * p.lddx + c);
                    f[i] = cols_load<W>(p, p.f + r * p.ldf + c);
                    jf[i] = p.post ? load_const(p, p.inv_f + r) : 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < B; ++i) {
                if (r0 + i >= rows) break;
                const bool start = r0 + i == 0;
                if (POST && p.gate) {
                    if (gate_left == 0) {
                        gate_row += p.ldgate;
                        gate_left = p.gate_rows;
                        gate = cols_load<W>(p, gate_row);
                    }
                    --gate_left;
                }
#pragma unroll
                for (int t = 0; t < W; ++t) {
                    if constexpr (PRE) {
                        const float v = __fmul_rn(d[i].v[t], __fmul_rn(y[i].v[t], iy[i]));
                        s_pre.v[t] = start ? v : __fadd_rn(s_pre.v[t], v);
                    }
                    if constexpr (POST || GATE) {
                        const float dt = __fmul_rn(dx[i].v[t], p.alpha);
                        const float fh = p.post ? __fmul_rn(f[i].v[t], jf[i]) : f[i].v[t];
                        if constexpr (POST) {
                            const float v = __fmul_rn(p.gate ? __fmul_rn(dt, gate.v[t]) : dt, fh);
                            s_post.v[t] = start ? v : __fadd_rn(s_post.v[t], v);
                        }
                        if constexpr (GATE) {
                            const float v = __fmul_rn(dt, p.post ? __fmul_rn(fh, post.v[t]) : fh);
                            s_gate.v[t] = start ? v : __fadd_rn(s_gate.v[t], v);
                        }
                    }
                }
            }
        }
        if constexpr (PRE) cols_store<W>(p, a.pre + run * p.n + c, s_pre);
        if constexpr (POST) cols_store<W>(p, a.post + run * p.n + c, s_post);
        if constexpr (GATE) cols_store<W>(p, a.gate + run * a.ldg + c, s_gate);
    }
}

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
__global__ void __launch_bounds__(1024) edge_fold_kernel(FoldArgs a) {
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

// ------------------------------------------------------------------- host ----

bool vec_row(const void *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 4 == 0; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int64_t pad4(int64_t n) { return (n + 3) / 4 * 4; }

// The column sums' scratch in floats, each array starting on 16 bytes: two
// columns of 1/rms, the run results of the two gains, those of the gate (none
// where a gate row has a single run: that run's result is the gradient), and
// further levels where a block has more than 1024 runs.
struct Scratch {
    int64_t runs;                   // run results of a gain
    int64_t gate_per, gate_runs;    // runs of one gate row; run results kept for the gate
    int64_t level;                  // rows of the further levels
    int64_t n4;
    uint64_t floats(int64_t rows) const {
        return uint64_t(2 * pad4(rows)) + uint64_t(2 * runs + gate_runs + level) * uint64_t(n4);
    }
};

Scratch scratch_plan(int64_t rows, int64_t cols, int64_t gates) {
    Scratch s;
    s.n4 = pad4(cols);
    s.runs = ceil_div(rows, RUN);
    s.gate_per = gates > 0 ? ceil_div(rows / gates, RUN) : 0;
    s.gate_runs = s.gate_per > 1 ? gates * s.gate_per : 0;
    // a level of r run results has at most r/32 + 1 a block, the blocks have
    // more than 1024 each, and each level is a 32nd of the one below: under
    // 1.1 * r/32 + 8 for each of three sums
    const int64_t most = std::max(s.runs > MAX_FOLD_ROWS ? s.runs : 0, s.gate_per > MAX_FOLD_ROWS ? s.gate_runs : 0);
    s.level = most ? 4 * ceil_div(most, RUN) + 64 : 0;
    return s;
}

// Scratch of a call: the caller's, or the library's pool.
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

// One CTA an SM at most (a CTA's teams fill it), a row a team at least.
template <class Kern, class Args>
int launch_teams(Kern kern, int threads, size_t smem, const Args &a, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return set_cuda_error(e);
    DeviceInfo di;
    const int64_t sms = current_device_info(&di) == REPOPS_OK ? di.sms : 152;
    kern<<<unsigned(std::min(a.rows, sms)), threads, smem, s>>>(a);
    return check_launch();
}

// Resident CTAs an SM of the forward kernel, asked for once a device (0: not
// yet): the question costs a quarter of the host's time in a call for one row.
// The kernel's shared-memory limit belongs to the context and is set each time
// where the default (48 KB) does not do.
template <int T, int KS, bool VEC>
int launch_forward_t(const EdgeArgs &a, cudaStream_t s) {
    constexpr size_t smem = size_t(T) * KS * 16 * (kEdgePrefetch<T> ? 4 : 2);
    static std::atomic<int> resident[64];
    DeviceInfo di;
    int rc = current_device_info(&di);
    if (rc != REPOPS_OK) return rc;
    auto kern = edge_forward_kernel<T, KS, VEC>;
    int per_sm = resident[di.device].load(std::memory_order_relaxed);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return set_cuda_error(e);
    }
    if (per_sm == 0) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, T, smem);
        if (e != cudaSuccess) return set_cuda_error(e);
        per_sm = std::max(per_sm, 1);
        resident[di.device].store(per_sm, std::memory_order_relaxed);
    }
    kern<<<unsigned(std::min<int64_t>(a.rows, int64_t(per_sm) * di.sms)), T, smem, s>>>(a);
    return check_launch();
}

template <bool VEC>
int launch_forward(const EdgeArgs &a, cudaStream_t s) {
    if (a.n <= 256) return launch_forward_t<32, 2, VEC>(a, s);
    if (a.n <= 512) return launch_forward_t<32, 4, VEC>(a, s);
    if (a.n <= 1024) return launch_forward_t<32, 8, VEC>(a, s);
    if (a.n <= 2048) return launch_forward_t<64, 8, VEC>(a, s);
    if (a.n <= 4096) return launch_forward_t<128, 8, VEC>(a, s);
    return launch_forward_t<256, 8, VEC>(a, s);
}

size_t long_row_smem(int64_t n) {
    const int64_t runs = ceil_div(n, RUN);
    return size_t(runs + ceil_div(runs, RUN)) * sizeof(float);
}

template <class Kern, class Args>
int launch_long(Kern kern, const Args &a, int64_t rows, int64_t n, cudaStream_t s) {
    const size_t smem = long_row_smem(n);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return set_cuda_error(e);
    kern<<<grid_for_rows(rows), 256, smem, s>>>(a);
    return check_launch();
}

template <int T, int KS, bool VEC, bool Q8, bool F>
int launch_rows_t(const EdgeBackArgs &a, cudaStream_t s) {
    constexpr int teams = kBackTeams<T, KS, F>;
    return launch_teams(edge_backward_kernel<T, KS, VEC, Q8, F>, T * teams,
                        F ? kTeamSmem<T, KS, 4, 3, teams> : kTeamSmem<T, KS, 3, 1, teams>, a, s);
}

template <bool VEC, bool Q8, bool F>
int launch_rows(const EdgeBackArgs &a, cudaStream_t s) {
    if (a.n <= 256) return launch_rows_t<32, 2, VEC, Q8, F>(a, s);
    if (a.n <= 512) return launch_rows_t<32, 4, VEC, Q8, F>(a, s);
    if (a.n <= 1024) return launch_rows_t<32, 8, VEC, Q8, F>(a, s);
    if (a.n <= 2048) return launch_rows_t<64, 8, VEC, Q8, F>(a, s);
    if (a.n <= 4096) return launch_rows_t<128, 8, VEC, Q8, F>(a, s);
    return launch_rows_t<256, 8, VEC, Q8, F>(a, s);
}

template <bool Q8, bool F>
int launch_columns(const ColArgs &a, bool vec, cudaStream_t s) {
    const int64_t threads = vec ? a.e.n / 4 : a.e.n;
    const dim3 grid(unsigned(ceil_div(threads, 128)), unsigned(std::min<int64_t>(a.runs, 65535)));
    auto go = [&](auto kern4, auto kern1) {
        if (vec) kern4<<<grid, 128, 0, s>>>(a);
        else kern1<<<grid, 128, 0, s>>>(a);
        return check_launch();
    };
#define REPOPS_COLUMNS(PRE, POST, GATE) \
    go(edge_columns_kernel<4, Q8, PRE, POST, GATE>, edge_columns_kernel<1, Q8, PRE, POST, GATE>)
    if constexpr (!F) return REPOPS_COLUMNS(true, false, false);
    else if (a.pre && a.post) return a.gate ? REPOPS_COLUMNS(true, true, true) : REPOPS_COLUMNS(true, true, false);
    else if (a.pre) return a.gate ? REPOPS_COLUMNS(true, false, true) : REPOPS_COLUMNS(true, false, false);
    else if (a.post) return a.gate ? REPOPS_COLUMNS(false, true, true) : REPOPS_COLUMNS(false, true, false);
    else return REPOPS_COLUMNS(false, false, true);
#undef REPOPS_COLUMNS
}

// The row kernel, the column terms and their folds.  dpre, dpost: n floats;
// dgate: gates x n at pitch lddgate; null where there is none.
template <bool Q8, bool F>
int run_backward(EdgeBackArgs e, float *dpre, float *dpost, float *dgate, int64_t lddgate, float *ws, bool vec,
                 cudaStream_t s) {
    const int64_t gates = dgate ? e.rows / e.gate_rows : 0;
    const Scratch sc = scratch_plan(e.rows, e.n, gates);
    e.inv_y = ws;
    e.inv_f = e.inv_y + pad4(e.rows);
    float *part = e.inv_f + pad4(e.rows);
    float *ppre = part, *ppost = ppre + sc.runs * sc.n4, *pgate = ppost + sc.runs * sc.n4;
    float *level = pgate + sc.gate_runs * sc.n4;
    int rc;
    if (e.n > MAX_STAGED_COLS) rc = launch_long(edge_backward_long_kernel<Q8, F>, e, e.rows, e.n, s);
    else if (vec) rc = launch_rows<true, Q8, F>(e, s);
    else rc = launch_rows<false, Q8, F>(e, s);
    if (rc != REPOPS_OK) return rc;
    if (!dpre && !dpost && !dgate) return REPOPS_OK;
    // a gate's runs coincide with the gains' where its rows are whole runs:
    // one pass makes all three sums
    float *gate_out = sc.gate_per == 1 ? dgate : pgate;
    const int64_t gate_ld = sc.gate_per == 1 ? lddgate : e.n;
    const bool together = dgate && (dpre || dpost) && (gates == 1 || e.gate_rows % RUN == 0);
    if (dpre || dpost) {
        const ColArgs c{e, e.rows, sc.runs, sc.runs, dpre ? ppre : nullptr, dpost ? ppost : nullptr,
                        together ? gate_out : nullptr, gate_ld};
        rc = launch_columns<Q8, F>(c, vec, s);
        if (rc != REPOPS_OK) return rc;
    }
    if (dgate && !together) {
        const ColArgs c{e, e.gate_rows, sc.gate_per, gates * sc.gate_per, nullptr, nullptr, gate_out, gate_ld};
        rc = launch_columns<Q8, F>(c, vec, s);
        if (rc != REPOPS_OK) return rc;
    }
    FoldArgs f{e};
    f.n = e.n;
    int sets = 0;
    int64_t blocks = 1, most = 1;
    auto add = [&](const float *in, float *out, int64_t nb, int64_t runs, int64_t ldo) {
        // one further level first for more than 1024 run results (twice for
        // more than 32768 of them, and so on): a column sum's pass per block
        while (rc == REPOPS_OK && runs > MAX_FOLD_ROWS) {
            const int64_t up = ceil_div(runs, RUN);
            const dim3 grid(unsigned(std::min<int64_t>(ceil_div(e.n, 256), 64)), unsigned(std::min<int64_t>(up, 65535)));
            for (int64_t b = 0; b < nb && rc == REPOPS_OK; ++b) {
                colsum_pass_kernel<<<grid, 256, 0, s>>>(runs, e.n, in + b * runs * e.n, e.n, level + b * up * e.n, e.n, e);
                rc = check_launch();
            }
            in = level;
            level += nb * up * sc.n4;
            runs = up;
        }
        f.s[sets++] = FoldSet{in, out, nb, runs, ldo};
        blocks = std::max(blocks, nb);
        most = std::max(most, runs);
    };
    if (dpre) add(ppre, dpre, 1, sc.runs, e.n);
    if (dpost) add(ppost, dpost, 1, sc.runs, e.n);
    if (dgate && sc.gate_per > 1) add(pgate, dgate, gates, sc.gate_per, lddgate);
    if (rc != REPOPS_OK || sets == 0) return rc;
    const dim3 grid(unsigned(ceil_div(e.n, RUN)), unsigned(std::min<int64_t>(blocks, 65535)), unsigned(sets));
    return launch_behind(edge_fold_kernel, grid, unsigned(ceil_div(most, RUN) * 32), 0, s, f);
}

}  // namespace
}  // namespace repops

using namespace repops;

namespace {

struct Span {
    const void *p;
    uint64_t bytes;
};

bool overlaps_any(Span o, std::initializer_list<Span> others) {
    if (!o.p) return false;
    for (const Span &t : others)
        if (t.p && ranges_overlap(o.p, o.bytes, t.p, t.bytes)) return true;
    return false;
}

bool too_long(int64_t cols) { return ceil_div(cols, RUN) > MAX_GENERIC_RUNS; }

}  // namespace

extern "C" int repops_rmsnorm_residual_f32(int64_t rows, int64_t cols, const float *x, int64_t ldx, const float *f,
                                           int64_t ldf, const float *post_gain, const float *gate, int64_t ldgate,
                                           int64_t gate_rows, float alpha, const float *pre_gain, float eps, float *y,
                                           int64_t ldy, float *h, int64_t ldh, cudaStream_t stream) {
    if (rows < 0 || cols < 0) return REPOPS_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return REPOPS_OK;
    if (!x || !f || !y || (pre_gain != nullptr) != (h != nullptr)) return REPOPS_ERR_INVALID_ARG;
    if (gate && (gate_rows < 1 || rows % gate_rows != 0)) return REPOPS_ERR_INVALID_ARG;
    if (too_long(cols)) return REPOPS_ERR_UNSUPPORTED;
    uint64_t xb, fb, yb, hb = 0, gb = 0;
    if (!rows_span(rows, cols, ldx, &xb) || !rows_span(rows, cols, ldf, &fb) || !rows_span(rows, cols, ldy, &yb) ||
        (h && !rows_span(rows, cols, ldh, &hb)) || (gate && !rows_span(rows / gate_rows, cols, ldgate, &gb)))
        return REPOPS_ERR_INVALID_ARG;
    // a row is read before either output of it is written: y or h may be x or
    // f themselves (the same pitch), but not both the same
    const uint64_t vb = uint64_t(cols) * 4u;
    const struct { float *p; uint64_t b; int64_t ld; } outs[2] = {{y, yb, ldy}, {h, hb, ldh}};
    for (const auto &o : outs) {
        if (!o.p) continue;
        if (overlaps_any({o.p, o.b}, {{post_gain, vb}, {gate, gb}, {pre_gain, vb}})) return REPOPS_ERR_ALIAS;
        if (!(o.p == x && o.ld == ldx) && ranges_overlap(o.p, o.b, x, xb)) return REPOPS_ERR_ALIAS;
        if (!(o.p == f && o.ld == ldf) && ranges_overlap(o.p, o.b, f, fb)) return REPOPS_ERR_ALIAS;
    }
    if (h && ranges_overlap(y, yb, h, hb)) return REPOPS_ERR_ALIAS;
    EdgeArgs a{{}, rows, cols, x, f, ldx, ldf, post_gain, gate, pre_gain, ldgate, gate ? gate_rows : 1, alpha, eps,
               y, h, ldy, ldh};
    a.reads(x, xb);
    a.reads(f, fb);
    a.reads(post_gain, vb);
    a.reads(gate, gb);
    a.reads(pre_gain, vb);
    a.writes(y, yb);
    a.writes(h, hb);
    if (const int rc = a.arm(); rc != REPOPS_OK) return rc;
    if (cols > MAX_STAGED_COLS) return launch_long(edge_forward_long_kernel, a, rows, cols, stream);
    const bool vec = cols % 4 == 0 && vec_row(x, ldx) && vec_row(f, ldf) && vec_row(y, ldy) && (!h || vec_row(h, ldh)) &&
                     vec_row(post_gain, 0) && vec_row(pre_gain, 0) && (!gate || vec_row(gate, ldgate));
    return vec ? launch_forward<true>(a, stream) : launch_forward<false>(a, stream);
}

extern "C" uint64_t repops_rmsnorm_residual_backward_workspace_bytes(int64_t rows, int64_t cols, int64_t gates) {
    if (rows <= 0 || cols <= 0 || gates < 0 || (gates > 0 && rows % gates != 0) || rows > (int64_t(1) << 40) ||
        cols > (int64_t(1) << 24))
        return 0;
    return scratch_plan(rows, cols, gates).floats(rows) * 4u;
}

extern "C" int repops_rmsnorm_residual_backward_f32(
    int64_t rows, int64_t cols, const float *dy, int64_t lddy, const float *dh, int64_t lddh, const float *y,
    int64_t ldy, const float *f, int64_t ldf, const float *post_gain, const float *gate, int64_t ldgate,
    int64_t gate_rows, float alpha, const float *pre_gain, float eps, float *dx, int64_t lddx, float *df,
    int64_t lddf, float *dpre, float *dpost, float *dgate, int64_t lddgate, void *ws, uint64_t ws_bytes,
    cudaStream_t stream) {
    if (rows < 0 || cols < 0) return REPOPS_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return REPOPS_OK;
    const bool pre = pre_gain != nullptr;
    if (!f || !dx || !df || (!dy && !dh) || pre != (dh != nullptr) || pre != (y != nullptr) ||
        pre != (dpre != nullptr) || (post_gain != nullptr) != (dpost != nullptr) ||
        (gate != nullptr) != (dgate != nullptr))
        return REPOPS_ERR_INVALID_ARG;
    if (gate && (gate_rows < 1 || rows % gate_rows != 0)) return REPOPS_ERR_INVALID_ARG;
    if (too_long(cols)) return REPOPS_ERR_UNSUPPORTED;
    const int64_t gates = gate ? rows / gate_rows : 0;
    uint64_t dyb = 0, dhb = 0, yb = 0, fb, gb = 0, dxb, dfb, dgb = 0;
    if ((dy && !rows_span(rows, cols, lddy, &dyb)) || (dh && !rows_span(rows, cols, lddh, &dhb)) ||
        (y && !rows_span(rows, cols, ldy, &yb)) || !rows_span(rows, cols, ldf, &fb) ||
        (gate && (!rows_span(gates, cols, ldgate, &gb) || !rows_span(gates, cols, lddgate, &dgb))) ||
        !rows_span(rows, cols, lddx, &dxb) || !rows_span(rows, cols, lddf, &dfb))
        return REPOPS_ERR_INVALID_ARG;
    const uint64_t vb = uint64_t(cols) * 4u, need = repops_rmsnorm_residual_backward_workspace_bytes(rows, cols, gates);
    // dx may be dy itself; the column sums read the other inputs after the
    // rows have been written
    const Span in_dy{dx == dy && lddx == lddy ? nullptr : dy, dyb};
    const Span outs[5] = {{dx, dxb}, {df, dfb}, {dpre, vb}, {dpost, vb}, {dgate, dgb}};
    for (int i = 0; i < 5; ++i) {
        if (overlaps_any(outs[i], {i == 0 ? in_dy : Span{dy, dyb}, {dh, dhb}, {y, yb}, {f, fb}, {post_gain, vb},
                                   {gate, gb}, {pre_gain, vb}, {ws, ws ? ws_bytes : 0}}))
            return REPOPS_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps_any(outs[i], {outs[j]})) return REPOPS_ERR_ALIAS;
    }
    if (need == 0) return REPOPS_ERR_UNSUPPORTED;
    if (overlaps_any({ws, ws ? ws_bytes : 0}, {{dy, dyb}, {dh, dhb}, {y, yb}, {f, fb}, {post_gain, vb}, {gate, gb},
                                               {pre_gain, vb}}))
        return REPOPS_ERR_ALIAS;
    Workspace w;
    int rc = w.get(ws, ws_bytes, need, stream);
    if (rc != REPOPS_OK) return rc;
    EdgeBackArgs e{};
    e.rows = rows; e.n = cols;
    e.y = y; e.ldy = ldy;
    e.dh = dh; e.lddh = lddh; e.dy = dy; e.lddy = lddy;
    e.pre = pre_gain;
    e.f = f; e.ldf = ldf;
    e.post = post_gain; e.gate = gate; e.ldgate = ldgate; e.gate_rows = gate ? gate_rows : 1;
    e.alpha = alpha; e.eps = eps;
    e.dx = dx; e.lddx = lddx; e.df = df; e.lddf = lddf;
    e.reads(dy, dyb);
    e.reads(dh, dhb);
    e.reads(y, yb);
    e.reads(f, fb);
    e.reads(post_gain, vb);
    e.reads(gate, gb);
    e.reads(pre_gain, vb);
    e.writes(dx, dxb);
    e.writes(df, dfb);
    e.writes(dpre, vb);
    e.writes(dpost, vb);
    e.writes(dgate, dgb);
    e.writes(w.p, need);
    if (rc = e.arm(); rc != REPOPS_OK) return w.release(rc);
    const bool vec = cols % 4 == 0 && (!dy || vec_row(dy, lddy)) && (!dh || vec_row(dh, lddh)) &&
                     (!y || vec_row(y, ldy)) && vec_row(f, ldf) && vec_row(post_gain, 0) && vec_row(pre_gain, 0) &&
                     (!gate || (vec_row(gate, ldgate) && vec_row(dgate, lddgate))) && vec_row(dx, lddx) &&
                     vec_row(df, lddf);
    return w.release(run_backward<false, true>(e, dpre, dpost, dgate, lddgate, w.p, vec, stream));
}

extern "C" uint64_t repops_rmsnorm_backward_i8_workspace_bytes(int64_t rows, int64_t cols) {
    return repops_rmsnorm_residual_backward_workspace_bytes(rows, cols, 0);
}

extern "C" int repops_rmsnorm_backward_i8(int64_t rows, int64_t cols, const int8_t *x, int64_t ldx,
                                          const float *x_scale, int64_t lds, int64_t group, const float *gamma,
                                          float eps, const float *dy, int64_t lddy, const float *res, int64_t ldres,
                                          float *dx, int64_t lddx, float *h, int64_t ldh, float *dgamma, void *ws,
                                          uint64_t ws_bytes, cudaStream_t stream) {
    if (rows < 0 || cols < 0 || !known_group(group)) return REPOPS_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return REPOPS_OK;
    if (!x || !x_scale || !gamma || !dy || !dx || !dgamma) return REPOPS_ERR_INVALID_ARG;
    if (too_long(cols)) return REPOPS_ERR_UNSUPPORTED;
    uint64_t xb, sb, dyb, rb = 0, dxb, hb = 0;
    if (!span_bytes(rows, cols, ldx, 1, &xb) || !span_bytes(rows, group_count(cols, group), lds, 4, &sb) ||
        !rows_span(rows, cols, lddy, &dyb) || (res && !rows_span(rows, cols, ldres, &rb)) ||
        !rows_span(rows, cols, lddx, &dxb) || (h && !rows_span(rows, cols, ldh, &hb)))
        return REPOPS_ERR_INVALID_ARG;
    const uint64_t vb = uint64_t(cols) * 4u, need = repops_rmsnorm_backward_i8_workspace_bytes(rows, cols);
    const Span in_res{dx == res && lddx == ldres ? nullptr : res, rb};
    const Span outs[3] = {{dx, dxb}, {h, hb}, {dgamma, vb}};
    for (int i = 0; i < 3; ++i) {
        if (overlaps_any(outs[i], {{x, xb}, {x_scale, sb}, {gamma, vb}, {dy, dyb}, i == 0 ? in_res : Span{res, rb},
                                   {ws, ws ? ws_bytes : 0}}))
            return REPOPS_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps_any(outs[i], {outs[j]})) return REPOPS_ERR_ALIAS;
    }
    if (need == 0) return REPOPS_ERR_UNSUPPORTED;
    if (overlaps_any({ws, ws ? ws_bytes : 0}, {{x, xb}, {x_scale, sb}, {gamma, vb}, {dy, dyb}, {res, rb}}))
        return REPOPS_ERR_ALIAS;
    Workspace w;
    int rc = w.get(ws, ws_bytes, need, stream);
    if (rc != REPOPS_OK) return rc;
    EdgeBackArgs e{};
    e.rows = rows; e.n = cols;
    e.q = x; e.ldq = ldx; e.s = x_scale; e.lds = lds; e.shift = group_shift(group);
    e.dh = dy; e.lddh = lddy; e.dy = res; e.lddy = ldres;
    e.pre = gamma;
    e.gate_rows = 1;
    e.eps = eps;
    e.dx = dx; e.lddx = lddx; e.h = h; e.ldh = ldh;
    e.reads(x, xb);
    e.reads(x_scale, sb);
    e.reads(gamma, vb);
    e.reads(dy, dyb);
    e.reads(res, rb);
    e.writes(dx, dxb);
    e.writes(h, hb);
    e.writes(dgamma, vb);
    e.writes(w.p, need);
    if (rc = e.arm(); rc != REPOPS_OK) return w.release(rc);
    const bool vec = cols % 4 == 0 && reinterpret_cast<uintptr_t>(x) % 4 == 0 && ldx % 4 == 0 && vec_row(gamma, 0) &&
                     vec_row(dy, lddy) && (!res || vec_row(res, ldres)) && vec_row(dx, lddx) &&
                     (!h || vec_row(h, ldh));
    return w.release(run_backward<true, false>(e, dgamma, nullptr, nullptr, 0, w.p, vec, stream));
}
