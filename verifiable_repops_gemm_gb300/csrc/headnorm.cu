// headnorm.cu -- RMSNorm of every query and key head and the position rotation in
// the same pass, with its backward; either may be left out, so this is the rotation
// of adjacent pairs or of halves, of a whole head or its first columns, at positions
// given for each row, as well.
//
// A head's values, each step one binary32 rounding (the separate operators' bits):
//   v = fl(fl(x * inv) * gain[j]), inv of repops_rmsnorm_rows_f32 over the head
//   pair i of the first 2 * pairs columns, (2i, 2i + 1) or (i, i + pairs):
//   (fl(fl(a*c) - fl(b*s)), fl(fl(a*s) + fl(b*c))), c and s of the row's position
// narrowed once.  The backward turns dy back, then as repops_rmsnorm_backward_f32;
// the gains' gradients are column sums over (row, head) in order.
//
// Bound by memory: x in and y out (dy and x in, dx out).  A head's sum is a tree
// whose first level folds 32 neighbouring values one after another, so heads pass
// through shared memory: neighbouring lanes copy neighbouring chunks, then a lane
// folds a run (the swizzle of rowtree.cuh serves both without conflicts), then
// neighbouring lanes write neighbouring chunks.  The backward's CTA takes 32 heads of
// one gain, a run of the gain's column sum, and so leaves a 32nd of the terms as
// run results instead of writing them all.
#include <algorithm>

#include "colfold.cuh"
#include "storage.cuh"

namespace repops {
namespace {

constexpr int kThreads = 256;
constexpr int kMostDim = 512;
constexpr float kNaN = __builtin_nanf("");

struct HeadArgs : DbgAccess {
    int64_t rows;
    int q, k, dim, pairs;
    int halves, inverse;
    const void *x;
    int64_t ldx;
    const void *dy;                  // backward
    int64_t lddy;
    void *y;                         // or dx
    int64_t ldy;
    const float *q_gain, *k_gain;
    float eps;
    const float *cosv, *sinv;
    int64_t positions;
    const void *pos;                 // a position a row, or null: first + row % period
    int pos_wide;
    int64_t first, period;
    float *part[2];                  // backward: run results of the two gains
};

// Where a head lies and where it stands: offsets in elements, the row of the table
// (-1: the row is left alone, -2: past the table).
struct Unit {
    int64_t x, dy, y;
    int pos, key;
};

__device__ __forceinline__ Unit unit_of(const HeadArgs &a, int64_t row, int head) {
    int64_t p;
    if (!a.pos) p = a.first + row % a.period;
    else if (a.pos_wide) p = load_const(a, static_cast<const int64_t *>(a.pos) + row);
    else p = load_const(a, static_cast<const int *>(a.pos) + row);
    Unit u;
    u.x = row * a.ldx + int64_t(head) * a.dim;
    u.dy = row * a.lddy + int64_t(head) * a.dim;
    u.y = row * a.ldy + int64_t(head) * a.dim;
    u.pos = p < 0 ? -1 : !a.pairs ? 0 : p >= a.positions ? -2 : int(p);
    u.key = head >= a.q;
    return u;
}

// cos and sin of pair i at a position (NaN past the table).
__device__ __forceinline__ float2 turn(const HeadArgs &a, int pos, int i) {
    if (pos < 0) return make_float2(kNaN, kNaN);
    const int64_t at = int64_t(pos) * a.pairs + i;
    return make_float2(load_const(a, a.cosv + at), load_const(a, a.sinv + at));
}
__device__ __forceinline__ float4 table4(const HeadArgs &a, const float *t, int pos, int i) {
    if (pos < 0) return make_float4(kNaN, kNaN, kNaN, kNaN);
    return load_const(a, reinterpret_cast<const float4 *>(t + int64_t(pos) * a.pairs + i));
}

template <bool BACK>
__device__ __forceinline__ void rotate(float &u, float &v, float c, float s) {
    const float a = u, b = v;
    if constexpr (BACK) {
        u = __fadd_rn(__fmul_rn(a, c), __fmul_rn(b, s));
        v = __fsub_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    } else {
        u = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
        v = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
    }
}

// Four neighbouring values in adjacent pairs, the first of column 4 * chunk.
template <bool BACK>
__device__ __forceinline__ void rotate_adjacent(const HeadArgs &a, int pos, int chunk, float4 &v) {
    const int i = 2 * chunk;
    if (i < a.pairs) {
        const float2 t = turn(a, pos, i);
        rotate<BACK>(v.x, v.y, t.x, t.y);
    }
    if (i + 1 < a.pairs) {
        const float2 t = turn(a, pos, i + 1);
        rotate<BACK>(v.z, v.w, t.x, t.y);
    }
}
// Four pairs of two halves, the first of pair i.
template <bool BACK>
__device__ __forceinline__ void rotate_halves(const HeadArgs &a, int pos, int i, float4 &u, float4 &v) {
    const float4 c = table4(a, a.cosv, pos, i), s = table4(a, a.sinv, pos, i);
    rotate<BACK>(u.x, v.x, c.x, s.x);
    rotate<BACK>(u.y, v.y, c.y, s.y);
    rotate<BACK>(u.z, v.z, c.z, s.z);
    rotate<BACK>(u.w, v.w, c.w, s.w);
}
// Value j of a head alone; `at` gives any of the head's values.
template <bool BACK, class F>
__device__ __forceinline__ float rotate_one(const HeadArgs &a, int pos, int j, F at) {
    if (j >= 2 * a.pairs) return at(j);
    const bool second = a.halves ? j >= a.pairs : j & 1;
    const int i = a.halves ? j - (second ? a.pairs : 0) : j >> 1;
    float u = at(a.halves ? i : 2 * i), v = at(a.halves ? i + a.pairs : 2 * i + 1);
    const float2 t = turn(a, pos, i);
    rotate<BACK>(u, v, t.x, t.y);
    return second ? v : u;
}

// ------------------------------------------------------------- the stage ----

// Chunk c (four values) of a head whose runs start at run r0; value j alone.
__device__ __forceinline__ int chunk_at(int r0, int c) { return stage_slot(r0 + (c >> 3), c & 7); }
__device__ __forceinline__ int value_at(int r0, int j) { return 4 * chunk_at(r0, j >> 2) + (j & 3); }

// The fold of run `run` of n values: f(value, column in the head).
template <class F>
__device__ __forceinline__ float fold_run(const float4 *stage, int run, int first, int n, F f) {
    float acc;
    if (n == RUN) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float4 v = stage[stage_slot(run, c)];
            const int j = first + 4 * c;
            acc = c == 0 ? f(v.x, j) : __fadd_rn(acc, f(v.x, j));
            acc = __fadd_rn(acc, f(v.y, j + 1));
            acc = __fadd_rn(acc, f(v.z, j + 2));
            acc = __fadd_rn(acc, f(v.w, j + 3));
        }
    } else {
        const float *s = reinterpret_cast<const float *>(stage);
        acc = f(s[4 * stage_slot(run, 0)], first);
        for (int i = 1; i < n; ++i) acc = __fadd_rn(acc, f(s[4 * stage_slot(run, i >> 2) + (i & 3)], first + i));
    }
    return acc;
}

__device__ __forceinline__ float fold_head(const float *red, int runs) {
    float acc = red[0];
    for (int i = 1; i < runs; ++i) acc = __fadd_rn(acc, red[i]);
    return acc;
}
__device__ __forceinline__ float inv_rms(float sum, float n, float eps) {
    return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sum, n), eps)));
}

__device__ __forceinline__ float4 scale4(float4 v, float f) {
    return make_float4(__fmul_rn(v.x, f), __fmul_rn(v.y, f), __fmul_rn(v.z, f), __fmul_rn(v.w, f));
}
__device__ __forceinline__ float4 mul4(float4 v, float4 f) {
    return make_float4(__fmul_rn(v.x, f.x), __fmul_rn(v.y, f.y), __fmul_rn(v.z, f.z), __fmul_rn(v.w, f.w));
}
__device__ __forceinline__ float4 gain4(const HeadArgs &a, int key, int c) {
    return load_const(a, reinterpret_cast<const float4 *>(key ? a.k_gain : a.q_gain) + c);
}

size_t stage_bytes(int units, int runs) { return size_t(units) * runs * RUN * 4; }

// ---------------------------------------------------------------- forward ----

// `units` heads a CTA, in the order of rows and heads.  VEC: four values an access
// everywhere.  NORM off: the rotation alone (BACK: its transpose), nothing staged
// but by the halves of pairs.
template <int TY, bool VEC, bool NORM, bool BACK>
__global__ void __launch_bounds__(kThreads) head_forward_kernel(const HeadArgs a, int units, int runs) {
    extern __shared__ __align__(16) float4 stage[];
    float *flat = reinterpret_cast<float *>(stage);
    float *red = flat + size_t(units) * runs * RUN;             // units x runs, then 1/rms
    Unit *info = reinterpret_cast<Unit *>(red + (units * runs + 1) / 2 * 2);
    const int heads = a.q + a.k;
    const int64_t total = a.rows * heads, u0 = blockIdx.x * int64_t(units);
    const int here = int(imin64(units, total - u0));
    for (int u = threadIdx.x; u < here; u += kThreads) {
        const int64_t row = (u0 + u) / heads;
        info[u] = unit_of(a, row, int(u0 + u - row * heads));
    }
    __syncthreads();
    const int chunks = a.dim / 4;
    if constexpr (VEC) {
        for (int i = threadIdx.x; i < here * chunks; i += kThreads) {
            const int u = i / chunks, c = i - u * chunks;
            stage[chunk_at(u * runs, c)] = load_four<TY>(a, a.x, info[u].x + 4 * c);
        }
    } else {
        for (int i = threadIdx.x; i < here * a.dim; i += kThreads) {
            const int u = i / a.dim, j = i - u * a.dim;
            flat[value_at(u * runs, j)] = load_one<TY>(a, a.x, info[u].x + j);
        }
    }
    __syncthreads();
    if constexpr (NORM) {
        for (int t = threadIdx.x; t < here * runs; t += kThreads) {
            const int first = (t % runs) * RUN;
            red[t] = fold_run(stage, t, first, min(RUN, a.dim - first), [](float v, int) { return __fmul_rn(v, v); });
        }
        __syncthreads();
        float inv = 0.0f;
        // at most one head a thread: a CTA has at least as many threads
        if (threadIdx.x < here) inv = inv_rms(fold_head(red + threadIdx.x * runs, runs), float(a.dim), a.eps);
        __syncthreads();
        if (threadIdx.x < here) red[threadIdx.x] = inv;
        __syncthreads();
    }
    if constexpr (VEC) {
        const int turned = a.halves ? a.pairs / 4 : 0, items = chunks - turned;
        for (int i = threadIdx.x; i < here * items; i += kThreads) {
            const int u = i / items, w = i - u * items;
            const Unit t = info[u];
            if (t.pos == -1) continue;
            const int c = w < turned ? w : w + turned;      // halves: the first half stands for both
            float4 v = stage[chunk_at(u * runs, c)];
            if constexpr (NORM) v = mul4(scale4(v, red[u]), gain4(a, t.key, c));
            if (w < turned) {
                float4 v2 = stage[chunk_at(u * runs, c + turned)];
                if constexpr (NORM) v2 = mul4(scale4(v2, red[u]), gain4(a, t.key, c + turned));
                rotate_halves<BACK>(a, t.pos, 4 * c, v, v2);
                store_four<TY>(a, a.y, t.y + 4 * (c + turned), v2);
            } else if (!a.halves) {
                rotate_adjacent<BACK>(a, t.pos, c, v);
            }
            store_four<TY>(a, a.y, t.y + 4 * c, v);
        }
    } else {
        for (int i = threadIdx.x; i < here * a.dim; i += kThreads) {
            const int u = i / a.dim, j = i - u * a.dim;
            const Unit t = info[u];
            if (t.pos == -1) continue;
            const float *gain = t.key ? a.k_gain : a.q_gain;
            const float v = rotate_one<BACK>(a, t.pos, j, [&](int c) {
                const float x = flat[value_at(u * runs, c)];
                return NORM ? __fmul_rn(__fmul_rn(x, red[u]), load_const(a, gain + c)) : x;
            });
            store_one<TY>(a, a.y, t.y + j, v);
        }
    }
}

// --------------------------------------------------------------- backward ----

// A run of 32 heads of one gain: the queries' runs first, then the keys'.
template <int TY, bool VEC>
__global__ void __launch_bounds__(kThreads) head_backward_kernel(const HeadArgs a, int64_t q_runs, int runs) {
    extern __shared__ __align__(16) float4 stage[];
    float4 *gs = stage + RUN * runs * 8;
    float *fx = reinterpret_cast<float *>(stage), *fg = reinterpret_cast<float *>(gs);
    float *red = fg + size_t(RUN) * runs * RUN;                  // 32 x runs
    float *inv = red + RUN * runs, *mean = inv + RUN;
    Unit *info = reinterpret_cast<Unit *>(mean + RUN);
    const int key = blockIdx.x >= q_runs;
    const int64_t run = blockIdx.x - (key ? q_runs : 0);
    const int heads = key ? a.k : a.q;
    const int64_t total = a.rows * heads, u0 = run * RUN;
    const int here = int(imin64(RUN, total - u0));
    if (int(threadIdx.x) < here) {
        const int64_t row = (u0 + threadIdx.x) / heads;
        info[threadIdx.x] = unit_of(a, row, int(u0 + threadIdx.x - row * heads) + (key ? a.q : 0));
    }
    __syncthreads();
    const float *gain = key ? a.k_gain : a.q_gain;
    const int chunks = a.dim / 4;
    if constexpr (VEC) {
        const int turned = a.halves ? a.pairs / 4 : 0, items = chunks - turned;
        const float4 zero = make_float4(0, 0, 0, 0);
        for (int i = threadIdx.x; i < here * items; i += kThreads) {
            const int u = i / items, w = i - u * items;
            const Unit t = info[u];
            const bool live = t.pos != -1;
            const int c = w < turned ? w : w + turned;
            float4 g = zero, x = zero;
            if (live) {
                g = load_four<TY>(a, a.dy, t.dy + 4 * c);
                x = load_four<TY>(a, a.x, t.x + 4 * c);
            }
            if (w < turned) {
                float4 g2 = zero, x2 = zero;
                if (live) {
                    g2 = load_four<TY>(a, a.dy, t.dy + 4 * (c + turned));
                    x2 = load_four<TY>(a, a.x, t.x + 4 * (c + turned));
                    rotate_halves<true>(a, t.pos, 4 * c, g, g2);
                }
                stage[chunk_at(u * runs, c + turned)] = x2;
                gs[chunk_at(u * runs, c + turned)] = g2;
            } else if (live && !a.halves) {
                rotate_adjacent<true>(a, t.pos, c, g);
            }
            stage[chunk_at(u * runs, c)] = x;
            gs[chunk_at(u * runs, c)] = g;
        }
    } else {
        for (int i = threadIdx.x; i < here * a.dim; i += kThreads) {
            const int u = i / a.dim, j = i - u * a.dim;
            const Unit t = info[u];
            float g = 0.0f, x = 0.0f;
            if (t.pos != -1) {
                x = load_one<TY>(a, a.x, t.x + j);
                g = rotate_one<true>(a, t.pos, j, [&](int c) { return load_one<TY>(a, a.dy, t.dy + c); });
            }
            fx[value_at(u * runs, j)] = x;
            fg[value_at(u * runs, j)] = g;
        }
    }
    __syncthreads();
    for (int t = threadIdx.x; t < here * runs; t += kThreads) {
        const int first = (t % runs) * RUN;
        red[t] = fold_run(stage, t, first, min(RUN, a.dim - first), [](float v, int) { return __fmul_rn(v, v); });
    }
    __syncthreads();
    if (int(threadIdx.x) < here)        // a row left alone adds +0, whatever eps
        inv[threadIdx.x] = info[threadIdx.x].pos == -1
                               ? 0.0f
                               : inv_rms(fold_head(red + threadIdx.x * runs, runs), float(a.dim), a.eps);
    __syncthreads();
    for (int t = threadIdx.x; t < here * runs; t += kThreads) {
        const int u = t / runs, first = (t - u * runs) * RUN;
        const float iv = inv[u];
        const float *g = fg;
        red[t] = fold_run(stage, t, first, min(RUN, a.dim - first), [&](float v, int j) {
            const float gy = __fmul_rn(g[value_at(u * runs, j)], load_const(a, gain + j));
            return __fmul_rn(gy, __fmul_rn(v, iv));
        });
    }
    __syncthreads();
    if (int(threadIdx.x) < here)
        mean[threadIdx.x] = __fdiv_rn(fold_head(red + threadIdx.x * runs, runs), float(a.dim));
    __syncthreads();
    auto grad = [&](float x, float g, float w, float iv, float m, float &term) {
        const float xh = __fmul_rn(x, iv);
        term = __fmul_rn(g, xh);
        return __fmul_rn(iv, __fsub_rn(__fmul_rn(g, w), __fmul_rn(xh, m)));
    };
    if constexpr (VEC) {
        for (int i = threadIdx.x; i < here * chunks; i += kThreads) {
            const int u = i / chunks, c = i - u * chunks, at = chunk_at(u * runs, c);
            const float4 x = stage[at], g = gs[at], w = load_const(a, reinterpret_cast<const float4 *>(gain) + c);
            const float iv = inv[u], m = mean[u];
            float4 d, t;
            d.x = grad(x.x, g.x, w.x, iv, m, t.x);
            d.y = grad(x.y, g.y, w.y, iv, m, t.y);
            d.z = grad(x.z, g.z, w.z, iv, m, t.z);
            d.w = grad(x.w, g.w, w.w, iv, m, t.w);
            gs[at] = t;
            if (info[u].pos != -1) store_four<TY>(a, a.y, info[u].y + 4 * c, d);
        }
    } else {
        for (int i = threadIdx.x; i < here * a.dim; i += kThreads) {
            const int u = i / a.dim, j = i - u * a.dim, at = value_at(u * runs, j);
            float t;
            const float d = grad(fx[at], fg[at], load_const(a, gain + j), inv[u], mean[u], t);
            fg[at] = t;
            if (info[u].pos != -1) store_one<TY>(a, a.y, info[u].y + j, d);
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < a.dim; j += kThreads) {
        float acc = fg[value_at(0, j)];
        for (int u = 1; u < here; ++u) acc = __fadd_rn(acc, fg[value_at(u * runs, j)]);
        store_global(a, a.part[key] + run * a.dim + j, acc);
    }
}

// ------------------------------------------------------------------- host ----

size_t forward_smem(int units, int runs) {
    return stage_bytes(units, runs) + size_t((units * runs + 1) / 2 * 2) * 4 + size_t(units) * sizeof(Unit);
}
size_t backward_smem(int runs) { return 2 * stage_bytes(RUN, runs) + size_t(RUN) * (runs + 2) * 4 + RUN * sizeof(Unit); }

template <int TY, bool VEC, bool NORM, bool BACK>
int launch_forward(const HeadArgs &a, cudaStream_t s) {
    DeviceInfo di;
    if (const int rc = current_device_info(&di); rc != REPOPS_OK) return rc;
    const int runs = int(ceil_div(a.dim, RUN));
    const int64_t total = a.rows * (a.q + a.k);
    // 16 KB of heads a CTA, fewer where there are too few to give every SM two CTAs
    const int units = int(std::max<int64_t>(1, std::min<int64_t>(128 / runs, ceil_div(total, 2 * di.sms))));
    if (ceil_div(total, units) > INT32_MAX) return REPOPS_ERR_UNSUPPORTED;
    head_forward_kernel<TY, VEC, NORM, BACK>
        <<<unsigned(ceil_div(total, units)), kThreads, forward_smem(units, runs), s>>>(a, units, runs);
    return check_launch();
}

template <int TY>
int forward_typed(const HeadArgs &a, bool vec, cudaStream_t s) {
    if (a.q_gain) return vec ? launch_forward<TY, true, true, false>(a, s) : launch_forward<TY, false, true, false>(a, s);
    if (a.inverse) return vec ? launch_forward<TY, true, false, true>(a, s) : launch_forward<TY, false, false, true>(a, s);
    return vec ? launch_forward<TY, true, false, false>(a, s) : launch_forward<TY, false, false, false>(a, s);
}

int forward_any(const HeadArgs &a, int type, bool vec, cudaStream_t s) {
    switch (type) {
        case REPOPS_TYPE_F32: return forward_typed<REPOPS_TYPE_F32>(a, vec, s);
        case REPOPS_TYPE_F16: return forward_typed<REPOPS_TYPE_F16>(a, vec, s);
        default: return forward_typed<REPOPS_TYPE_BF16>(a, vec, s);
    }
}

template <int TY, bool VEC>
int launch_backward(const HeadArgs &a, int64_t q_runs, int64_t k_runs, cudaStream_t s) {
    const int runs = int(ceil_div(a.dim, RUN));
    const size_t smem = backward_smem(runs);
    auto kern = head_backward_kernel<TY, VEC>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return set_cuda_error(e);
    }
    kern<<<unsigned(q_runs + k_runs), kThreads, smem, s>>>(a, q_runs, runs);
    return check_launch();
}

// Run results of a gain's sum, and those of its further level where there are more
// than the last fold takes (a 32nd of them, of more than 1024; twice and so on).
int64_t level_rows(int64_t runs) { return runs > MAX_FOLD_ROWS ? 2 * ceil_div(runs, RUN) + 8 : 0; }


// The checks both directions share; what they return is REPOPS_OK with sizes of
// nothing to do (rows or heads of 0), which the callers look at first.
int check_shape(int64_t rows, int64_t q, int64_t k, int64_t dim, int type) {
    if (rows < 0 || q < 0 || k < 0 || dim < 1 || !known_storage(type)) return REPOPS_ERR_INVALID_ARG;
    if (dim > kMostDim || q > 65536 || k > 65536 || rows > (int64_t(1) << 40)) return REPOPS_ERR_UNSUPPORTED;
    return REPOPS_OK;
}

int check_table(const HeadArgs &a, int64_t rows) {
    if (a.pairs < 0 || 2 * int64_t(a.pairs) > a.dim || (a.pos_wide != 0 && a.pos_wide != 1)) return REPOPS_ERR_INVALID_ARG;
    if (a.pairs && (!a.cosv || !a.sinv || a.positions < 1 || a.positions > INT64_MAX / 8 / a.pairs))
        return REPOPS_ERR_INVALID_ARG;
    if (a.positions > INT32_MAX) return REPOPS_ERR_UNSUPPORTED;
    if (!a.pos) {
        if (a.first < 0 || a.period < 1) return REPOPS_ERR_INVALID_ARG;
        if (a.pairs && a.first > a.positions - std::min(rows, a.period)) return REPOPS_ERR_INVALID_ARG;
    }
    return REPOPS_OK;
}

bool vec4(const void *p, int64_t ld, unsigned size) {
    return reinterpret_cast<uintptr_t>(p) % (4 * size) == 0 && ld % 4 == 0;
}

}  // namespace
}  // namespace repops

using namespace repops;

namespace {

struct Span {
    const void *p;
    uint64_t bytes;
};

bool overlaps(Span o, std::initializer_list<Span> others) {
    for (const Span &t : others)
        if (o.p && t.p && ranges_overlap(o.p, o.bytes, t.p, t.bytes)) return true;
    return false;
}

HeadArgs make_args(int64_t rows, int64_t q, int64_t k, int64_t dim, int64_t pairs, int layout, const float *q_gain,
                   const float *k_gain, float eps, const float *cosv, const float *sinv, int64_t positions,
                   const void *pos, int pos_wide, int64_t first, int64_t period) {
    HeadArgs a{};
    a.rows = rows;
    a.q = int(q);
    a.k = int(k);
    a.dim = int(dim);
    a.pairs = pairs >= 0 && pairs <= kMostDim ? int(pairs) : -1;
    a.halves = layout == REPOPS_ROPE_HALVES && pairs > 0;
    a.q_gain = q_gain;
    a.k_gain = k_gain;
    a.eps = eps;
    a.cosv = cosv;
    a.sinv = sinv;
    a.positions = positions;
    a.pos = pos;
    a.pos_wide = pos_wide;
    a.first = first;
    a.period = period;
    return a;
}

bool table_vec(const HeadArgs &a) {
    return a.dim % 4 == 0 && (!a.halves || (a.pairs % 4 == 0 && reinterpret_cast<uintptr_t>(a.cosv) % 16 == 0 &&
                                            reinterpret_cast<uintptr_t>(a.sinv) % 16 == 0)) &&
           reinterpret_cast<uintptr_t>(a.q_gain) % 16 == 0 && reinterpret_cast<uintptr_t>(a.k_gain) % 16 == 0;
}

}  // namespace

extern "C" int repops_head_norm_rope(int64_t rows, int64_t q_heads, int64_t k_heads, int64_t dim, const void *x,
                                     int type, int64_t ldx, const float *q_gain, const float *k_gain, float eps,
                                     const float *cos_tab, const float *sin_tab, int64_t pairs, int64_t positions,
                                     int layout, int inverse, const void *pos, int pos_wide, int64_t first,
                                     int64_t period, void *y, int64_t ldy, cudaStream_t stream) {
    if (const int rc = check_shape(rows, q_heads, k_heads, dim, type); rc != REPOPS_OK) return rc;
    if (layout != REPOPS_ROPE_ADJACENT && layout != REPOPS_ROPE_HALVES) return REPOPS_ERR_INVALID_ARG;
    const bool norm = q_gain || k_gain;
    if ((norm && inverse) || (norm && ((q_heads && !q_gain) || (k_heads && !k_gain)))) return REPOPS_ERR_INVALID_ARG;
    HeadArgs a = make_args(rows, q_heads, k_heads, dim, pairs, layout, norm && !q_gain ? k_gain : q_gain,
                           norm && !k_gain ? q_gain : k_gain, eps, cos_tab, sin_tab, positions, pos, pos_wide, first, period);
    if (const int rc = check_table(a, rows); rc != REPOPS_OK) return rc;
    const int64_t width = (q_heads + k_heads) * dim;
    const unsigned size = storage_size(type);
    uint64_t xb, yb;
    if (!span_bytes(rows, width, ldx, size, &xb) || !span_bytes(rows, width, ldy, size, &yb)) return REPOPS_ERR_INVALID_ARG;
    if (rows == 0 || width == 0) return REPOPS_OK;
    if (!x || !y || reinterpret_cast<uintptr_t>(x) % size != 0 || reinterpret_cast<uintptr_t>(y) % size != 0)
        return REPOPS_ERR_INVALID_ARG;
    const uint64_t tb = pairs ? uint64_t(positions) * uint64_t(pairs) * 4u : 0, gb = uint64_t(dim) * 4u,
                   pb = uint64_t(rows) * (pos_wide ? 8u : 4u);
    const Span out{y, yb};
    if (!(y == x && ldy == ldx) && overlaps(out, {{x, xb}})) return REPOPS_ERR_ALIAS;
    if (overlaps(out, {{pairs ? cos_tab : nullptr, tb}, {pairs ? sin_tab : nullptr, tb}, {q_gain, gb}, {k_gain, gb}, {pos, pb}}))
        return REPOPS_ERR_ALIAS;
    a.x = x;
    a.ldx = ldx;
    a.y = y;
    a.ldy = ldy;
    a.inverse = inverse != 0;
    a.reads(x, xb);
    a.reads(pairs ? cos_tab : nullptr, tb);
    a.reads(pairs ? sin_tab : nullptr, tb);
    a.reads(a.q_gain, gb);
    a.reads(a.k_gain, gb);
    a.reads(pos, pb);
    a.writes(y, yb);
    if (const int rc = a.arm(); rc != REPOPS_OK) return rc;
    return forward_any(a, type, table_vec(a) && vec4(x, ldx, size) && vec4(y, ldy, size), stream);
}

extern "C" uint64_t repops_head_norm_rope_backward_workspace_bytes(int64_t rows, int64_t q_heads, int64_t k_heads,
                                                                   int64_t dim) {
    if (check_shape(rows, q_heads, k_heads, dim, REPOPS_TYPE_F32) != REPOPS_OK) return 0;
    const int64_t q = ceil_div(rows * q_heads, RUN), k = ceil_div(rows * k_heads, RUN);
    return uint64_t(q + k + level_rows(q) + level_rows(k)) * uint64_t(ceil_div(dim, 4) * 4) * 4u;
}

extern "C" int repops_head_norm_rope_backward(int64_t rows, int64_t q_heads, int64_t k_heads, int64_t dim,
                                              const void *dy, int type, int64_t lddy, const void *x, int64_t ldx,
                                              const float *q_gain, const float *k_gain, float eps,
                                              const float *cos_tab, const float *sin_tab, int64_t pairs,
                                              int64_t positions, int layout, const void *pos, int pos_wide,
                                              int64_t first, int64_t period, void *dx, int64_t lddx, float *dq_gain,
                                              float *dk_gain, void *ws, uint64_t ws_bytes, cudaStream_t stream) {
    if (const int rc = check_shape(rows, q_heads, k_heads, dim, type); rc != REPOPS_OK) return rc;
    if (layout != REPOPS_ROPE_ADJACENT && layout != REPOPS_ROPE_HALVES) return REPOPS_ERR_INVALID_ARG;
    if ((q_heads > 0) != (q_gain != nullptr) || (k_heads > 0) != (k_gain != nullptr) ||
        (q_gain != nullptr) != (dq_gain != nullptr) || (k_gain != nullptr) != (dk_gain != nullptr))
        return REPOPS_ERR_INVALID_ARG;
    HeadArgs a = make_args(rows, q_heads, k_heads, dim, pairs, layout, q_gain, k_gain, eps, cos_tab, sin_tab, positions,
                           pos, pos_wide, first, period);
    if (const int rc = check_table(a, rows); rc != REPOPS_OK) return rc;
    const int64_t width = (q_heads + k_heads) * dim;
    const unsigned size = storage_size(type);
    uint64_t xb, dyb, dxb;
    if (!span_bytes(rows, width, ldx, size, &xb) || !span_bytes(rows, width, lddy, size, &dyb) ||
        !span_bytes(rows, width, lddx, size, &dxb))
        return REPOPS_ERR_INVALID_ARG;
    if (rows == 0 || width == 0) return REPOPS_OK;
    if (!x || !dy || !dx || reinterpret_cast<uintptr_t>(x) % size != 0 || reinterpret_cast<uintptr_t>(dy) % size != 0 ||
        reinterpret_cast<uintptr_t>(dx) % size != 0)
        return REPOPS_ERR_INVALID_ARG;
    const int64_t q_runs = ceil_div(rows * q_heads, RUN), k_runs = ceil_div(rows * k_heads, RUN);
    if (q_runs + k_runs > INT32_MAX) return REPOPS_ERR_UNSUPPORTED;
    const uint64_t tb = pairs ? uint64_t(positions) * uint64_t(pairs) * 4u : 0, gb = uint64_t(dim) * 4u,
                   pb = uint64_t(rows) * (pos_wide ? 8u : 4u),
                   need = repops_head_norm_rope_backward_workspace_bytes(rows, q_heads, k_heads, dim);
    const float *ct = pairs ? cos_tab : nullptr, *st = pairs ? sin_tab : nullptr;
    const Span ins[] = {{x, xb}, {ct, tb}, {st, tb}, {q_gain, gb}, {k_gain, gb}, {pos, pb}, {ws, ws ? ws_bytes : 0}};
    const Span outs[3] = {{dx, dxb}, {dq_gain, gb}, {dk_gain, gb}};
    for (int i = 0; i < 3; ++i) {
        for (const Span &in : ins)
            if (overlaps(outs[i], {in})) return REPOPS_ERR_ALIAS;
        // dx may be dy: a head is read before it is written
        if (!(i == 0 && dx == dy && lddx == lddy) && overlaps(outs[i], {{dy, dyb}})) return REPOPS_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], {outs[j]})) return REPOPS_ERR_ALIAS;
    }
    if (overlaps({ws, ws ? ws_bytes : 0}, {{x, xb}, {ct, tb}, {st, tb}, {q_gain, gb}, {k_gain, gb}, {pos, pb}, {dy, dyb}}))
        return REPOPS_ERR_ALIAS;
    Workspace w;
    if (const int rc = w.get(ws, ws_bytes, need, stream); rc != REPOPS_OK) return rc;
    a.x = x;
    a.ldx = ldx;
    a.dy = dy;
    a.lddy = lddy;
    a.y = dx;
    a.ldy = lddx;
    a.part[0] = w.p;
    a.part[1] = w.p + q_runs * dim;
    a.reads(x, xb);
    a.reads(dy, dyb);
    a.reads(ct, tb);
    a.reads(st, tb);
    a.reads(q_gain, gb);
    a.reads(k_gain, gb);
    a.reads(pos, pb);
    a.writes(dx, dxb);
    a.writes(dq_gain, gb);
    a.writes(dk_gain, gb);
    a.writes(w.p, need);
    int rc = a.arm();
    if (rc != REPOPS_OK) return w.release(rc);
    const bool vec = table_vec(a) && vec4(x, ldx, size) && vec4(dy, lddy, size) && vec4(dx, lddx, size);
    switch (type) {
        case REPOPS_TYPE_F32:
            rc = vec ? launch_backward<REPOPS_TYPE_F32, true>(a, q_runs, k_runs, stream)
                     : launch_backward<REPOPS_TYPE_F32, false>(a, q_runs, k_runs, stream);
            break;
        case REPOPS_TYPE_F16:
            rc = vec ? launch_backward<REPOPS_TYPE_F16, true>(a, q_runs, k_runs, stream)
                     : launch_backward<REPOPS_TYPE_F16, false>(a, q_runs, k_runs, stream);
            break;
        default:
            rc = vec ? launch_backward<REPOPS_TYPE_BF16, true>(a, q_runs, k_runs, stream)
                     : launch_backward<REPOPS_TYPE_BF16, false>(a, q_runs, k_runs, stream);
    }
    FoldArgs f{a};
    f.n = dim;
    float *level = a.part[1] + k_runs * dim;
    int sets = 0;
    int64_t most = 1;
    auto add = [&](const float *in, float *out, int64_t n) {
        while (rc == REPOPS_OK && n > MAX_FOLD_ROWS) {
            const int64_t up = ceil_div(n, RUN);
            const dim3 grid(unsigned(ceil_div(dim, 256)), unsigned(std::min<int64_t>(up, 65535)));
            colsum_pass_kernel<<<grid, 256, 0, stream>>>(n, dim, in, dim, level, dim, a);
            rc = check_launch();
            in = level;
            level += up * dim;
            n = up;
        }
        f.s[sets++] = FoldSet{in, out, 1, n, dim};
        most = std::max(most, n);
    };
    if (q_runs) add(a.part[0], dq_gain, q_runs);
    if (k_runs) add(a.part[1], dk_gain, k_runs);
    if (rc == REPOPS_OK)
        rc = launch_behind(column_fold_kernel, dim3(unsigned(ceil_div(dim, RUN)), 1, unsigned(sets)),
                           unsigned(ceil_div(most, RUN) * 32), 0, stream, f);
    return w.release(rc);
}
