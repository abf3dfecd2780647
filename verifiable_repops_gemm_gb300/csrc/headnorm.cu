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
// neighbouring lanes write neighbouring chunks.  A warp takes the heads of 32 runs (16
// of 64 columns) by itself, 4 KB, and no CTA waits for another warp's.  The backward's
// CTA takes 32 heads of one gain, a run of the gain's column sum, and so leaves a 32nd
// of the terms as run results instead of writing them all.
//
// Measured, 4096 rows of 32 query and 8 key heads of 64 in float32, a ninth of them
// without a position, graph-replayed: 20.7 us forward (24.8 with a CTA's heads in common
// and barriers between the phases), 39 us with the gains' gradients backward (47 with a
// CTA's in common, 42 with each head's loads behind the one's before); with all rows
// live 24.7 and 43 (3.4 and 2.9 TB/s), in bfloat16 22.5 and 41, the rotation alone 17.8
// and 16.5.  What bounds them now are the latencies of
// a warp's phases together with the issue of some 37 instructions a value forward and 65
// backward, most of them addresses, swizzles and the trees' additions one by one.
#include <algorithm>

#include "colfold.cuh"
#include "storage.cuh"

namespace repops {
namespace {

constexpr int kWarps = 4;            // of a forward CTA
constexpr int kMostDim = 512;
constexpr float kNaN = __builtin_nanf("");

// i / d for i < 2^16 and d <= 2^11 by one multiplication.
struct Divisor {
    int d;
    uint32_t magic;
};
inline Divisor divisor(int64_t d) { return {int(d), d > 1 ? uint32_t(((uint64_t(1) << 32) + uint64_t(d) - 1) / uint64_t(d)) : 0}; }
__device__ __forceinline__ int quotient(int i, const Divisor &d) { return d.d == 1 ? i : int(__umulhi(uint32_t(i), d.magic)); }

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
    Divisor runs;                    // runs of a head
    int units;                       // heads of a warp: 32 / runs
    int whole, per;                  // chunks (or values) of a head; those rotated together as one
    int whole_shift, per_shift;      // 2^shift lanes take a head's
};

// Where a head lies and where it stands: offsets in elements, the row of the table
// (-1: the row is left alone, -2: past the table).
struct alignas(16) Unit {
    int64_t x, y, dy;
    int pos, key;
};

__device__ __forceinline__ void place(const HeadArgs &a, Unit &u, int64_t row, int head) {
    u.x = row * a.ldx + int64_t(head) * a.dim;
    u.y = row * a.ldy + int64_t(head) * a.dim;
    u.dy = row * a.lddy + int64_t(head) * a.dim;
    u.key = head >= a.q;
}
__device__ __forceinline__ int position_of(const HeadArgs &a, int64_t row) {
    int64_t p;
    if (!a.pos) p = a.first + (row < a.period ? row : row % a.period);
    else if (a.pos_wide) p = load_const(a, static_cast<const int64_t *>(a.pos) + row);
    else p = load_const(a, static_cast<const int *>(a.pos) + row);
    return p < 0 ? -1 : !a.pairs ? 0 : p >= a.positions ? -2 : int(p);
}
// The row of head n of `heads` a row.
__device__ __forceinline__ int64_t row_of(int64_t n, int heads) {
    return n < (int64_t(1) << 32) ? int64_t(uint32_t(n) / uint32_t(heads)) : n / heads;
}

__device__ __forceinline__ float2 turn(const HeadArgs &a, int pos, int i) {
    if (pos < 0) return make_float2(kNaN, kNaN);
    const int64_t at = int64_t(pos) * a.pairs + i;
    return make_float2(load_const(a, a.cosv + at), load_const(a, a.sinv + at));
}

// The cos and sin of a lane's pairs, kept while the position stays the same: a warp's
// heads are of one row or two.
struct Turn {
    int pos = -3;
    float4 c, s;                     // halves: of pairs i .. i + 3; adjacent: of i and i + 1
    __device__ __forceinline__ void halves(const HeadArgs &a, int p, int i) {
        if (p == pos) return;
        pos = p;
        c = s = make_float4(kNaN, kNaN, kNaN, kNaN);         // past the table
        if (p < 0) return;
        const int64_t at = int64_t(p) * a.pairs + i;
        c = load_const(a, reinterpret_cast<const float4 *>(a.cosv + at));
        s = load_const(a, reinterpret_cast<const float4 *>(a.sinv + at));
    }
    __device__ __forceinline__ void adjacent(const HeadArgs &a, int p, int i) {
        if (p == pos) return;
        pos = p;
        float2 u = turn(a, p, i), v = make_float2(0.0f, 0.0f);
        if (i + 1 < a.pairs) v = turn(a, p, i + 1);
        c.x = u.x;
        s.x = u.y;
        c.y = v.x;
        s.y = v.y;
    }
};

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
__device__ __forceinline__ void rotate_adjacent(const HeadArgs &a, Turn &t, int pos, int chunk, float4 &v) {
    const int i = 2 * chunk;
    if (i >= a.pairs) return;
    t.adjacent(a, pos, i);
    rotate<BACK>(v.x, v.y, t.c.x, t.s.x);
    if (i + 1 < a.pairs) rotate<BACK>(v.z, v.w, t.c.y, t.s.y);
}
// Four pairs of two halves, the first of pair i.
template <bool BACK>
__device__ __forceinline__ void rotate_halves(const HeadArgs &a, Turn &t, int pos, int i, float4 &u, float4 &v) {
    t.halves(a, pos, i);
    rotate<BACK>(u.x, v.x, t.c.x, t.s.x);
    rotate<BACK>(u.y, v.y, t.c.y, t.s.y);
    rotate<BACK>(u.z, v.z, t.c.z, t.s.z);
    rotate<BACK>(u.w, v.w, t.c.w, t.s.w);
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

// The sum of the squares of run `run` of n values.  VEC: n is a multiple of four; with
// heads of whole runs no lane is asked where its run ends (heads of 80 otherwise: value
// by value the shorter runs' lanes cost 5% of the backward).
template <bool VEC>
__device__ __forceinline__ float fold_squares(const HeadArgs &a, const float4 *stage, int run, int n) {
    float acc = 0.0f;
    auto chunk = [&](int c) {
        const float4 v = stage[stage_slot(run, c)];
        acc = c == 0 ? __fmul_rn(v.x, v.x) : __fadd_rn(acc, __fmul_rn(v.x, v.x));
        acc = __fadd_rn(acc, __fmul_rn(v.y, v.y));
        acc = __fadd_rn(acc, __fmul_rn(v.z, v.z));
        acc = __fadd_rn(acc, __fmul_rn(v.w, v.w));
    };
    if (VEC && a.dim % RUN == 0) {
#pragma unroll
        for (int c = 0; c < 8; ++c) chunk(c);
    } else if (VEC) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (4 * c < n) chunk(c);
    } else {
        const float *s = reinterpret_cast<const float *>(stage);
        for (int i = 0; i < n; ++i) {
            const float v = s[4 * stage_slot(run, i >> 2) + (i & 3)], q = __fmul_rn(v, v);
            acc = i == 0 ? q : __fadd_rn(acc, q);
        }
    }
    return acc;
}

// The fold of a head's run results, which the lanes from u * runs on hold.
__device__ __forceinline__ float fold_head(const HeadArgs &a, float acc) {
    const int base = quotient(threadIdx.x & 31, a.runs) * a.runs.d;
    float sum = __shfl_sync(0xffffffffu, acc, base);
    for (int r = 1; r < a.runs.d; ++r) sum = __fadd_rn(sum, __shfl_sync(0xffffffffu, acc, base + r));
    return sum;
}
// Column of the first value of this lane's run in its head, and the run's length.
__device__ __forceinline__ int run_first(const HeadArgs &a) {
    const int lane = threadIdx.x & 31;
    return (lane - quotient(lane, a.runs) * a.runs.d) * RUN;
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

// A warp's heads: 32 runs of 32 values, and where the heads lie.
struct WarpHeads {
    float4 x[RUN * 8];
    Unit unit[RUN];
    float inv[RUN];
};

// f(head, w, kept) for w < per of every head u < here, 2^shift lanes to a head, so that a
// lane meets the same w in each, and what f keeps for it is its own.
template <class Kept, int UNROLL, class F>
__device__ __forceinline__ void each_part(int here, int per, int shift, F f) {
    const int lane = threadIdx.x & 31, sub = lane & ((1 << shift) - 1), from = lane >> shift, step = 32 >> shift;
    for (int w = sub; w < per; w += 1 << shift) {
        Kept kept;
#pragma unroll UNROLL
        for (int u = from; u < here; u += step) f(u, w, kept);
    }
}
struct Nothing {};

// ---------------------------------------------------------------- forward ----

// VEC: four values an access everywhere (20.7 us above, value by value 46.5; backward 39
// and 136).  NORM off: the rotation alone (BACK: its
// transpose).
template <int TY, bool VEC, bool NORM, bool BACK>
__global__ void __launch_bounds__(kWarps * 32, 10) head_forward_kernel(const HeadArgs a) {
    __shared__ WarpHeads heads[kWarps];
    WarpHeads &h = heads[threadIdx.x >> 5];
    float *flat = reinterpret_cast<float *>(h.x);
    const int lane = threadIdx.x & 31, runs = a.runs.d, per_row = a.q + a.k;
    const int64_t total = a.rows * per_row, u0 = (blockIdx.x * int64_t(kWarps) + (threadIdx.x >> 5)) * a.units;
    if (u0 >= total) return;
    const int here = int(imin64(a.units, total - u0));
    int pos_of = -1;
    if (lane < here) {
        const int64_t row = row_of(u0 + lane, per_row);
        place(a, h.unit[lane], row, int(u0 + lane - row * per_row));
        pos_of = position_of(a, row);
    }
    __syncwarp();
    // a head has `per` chunks (halves: pairs of chunks that are rotated together, and
    // the rest), or without VEC values
    const int turned = a.halves ? a.pairs / 4 : 0;
    if constexpr (VEC) {
        each_part<Nothing, 8>(here, a.whole, a.whole_shift, [&](int u, int c, Nothing &) {
            h.x[chunk_at(u * runs, c)] = load_four<TY>(a, a.x, h.unit[u].x + 4 * c);
        });
    } else {
        each_part<Nothing, 4>(here, a.whole, a.whole_shift, [&](int u, int j, Nothing &) {
            flat[value_at(u * runs, j)] = load_one<TY>(a, a.x, h.unit[u].x + j);
        });
    }
    if (lane < here) h.unit[lane].pos = pos_of;      // asked for before the values, wanted after them
    __syncwarp();
    if constexpr (NORM) {
        const int first = run_first(a);
        float acc = 0.0f;
        if (lane < here * runs)
            acc = fold_squares<VEC>(a, h.x, lane, min(RUN, a.dim - first));
        const float inv = inv_rms(fold_head(a, acc), float(a.dim), a.eps);
        if (first == 0) h.inv[quotient(lane, a.runs)] = inv;
        __syncwarp();
    }
    if constexpr (VEC) {
        struct Kept {
            Turn turn;
            int key = -1;
            float4 g, g2;
        };
        each_part<Kept, 1>(here, a.per, a.per_shift, [&](int u, int w, Kept &k) {
            const int c = w < turned ? w : w + turned;
            const int64_t y = h.unit[u].y;
            const int pos = h.unit[u].pos, key = h.unit[u].key;
            if (pos == -1) return;
            const float iv = NORM ? h.inv[u] : 0.0f;
            if (NORM && key != k.key) {
                k.key = key;
                k.g = gain4(a, key, c);
                if (w < turned) k.g2 = gain4(a, key, c + turned);
            }
            float4 v = h.x[chunk_at(u * runs, c)];
            if constexpr (NORM) v = mul4(scale4(v, iv), k.g);
            if (w < turned) {
                float4 v2 = h.x[chunk_at(u * runs, c + turned)];
                if constexpr (NORM) v2 = mul4(scale4(v2, iv), k.g2);
                rotate_halves<BACK>(a, k.turn, pos, 4 * c, v, v2);
                store_four<TY>(a, a.y, y + 4 * (c + turned), v2);
            } else if (!a.halves) {
                rotate_adjacent<BACK>(a, k.turn, pos, c, v);
            }
            store_four<TY>(a, a.y, y + 4 * c, v);
        });
    } else {
        each_part<Nothing, 1>(here, a.per, a.per_shift, [&](int u, int j, Nothing &) {
            const Unit t = h.unit[u];
            if (t.pos == -1) return;
            const float *gain = t.key ? a.k_gain : a.q_gain;
            const float v = rotate_one<BACK>(a, t.pos, j, [&](int c) {
                const float x = flat[value_at(u * runs, c)];
                return NORM ? __fmul_rn(__fmul_rn(x, h.inv[u]), load_const(a, gain + c)) : x;
            });
            store_one<TY>(a, a.y, t.y + j, v);
        });
    }
}

// --------------------------------------------------------------- backward ----

// A run of 32 heads of one gain: the queries' runs first, then the keys'.  Each warp
// takes the heads of 32 of its runs of columns; the terms of the gain's gradient
// replace the turned dy in shared memory, where the CTA folds them.
struct WarpHeadsBack {
    float4 *x, *g;                   // 32 runs of 32 values each
    Unit *unit;                      // where its heads lie; no more than there are: heads of
    float *inv, *mean;               // 64 leave room for 12 CTAs an SM so, for 11 with 32
};
constexpr size_t kStage = RUN * 8 * sizeof(float4);
__host__ __device__ constexpr size_t back_bytes(int units) {
    return 2 * kStage + (size_t(units) * (sizeof(Unit) + 2 * sizeof(float)) + 15) / 16 * 16;
}
constexpr size_t kMostBack = RUN / 2 * back_bytes(2);         // heads of more than 320: two a warp
__device__ __forceinline__ WarpHeadsBack back_heads(unsigned char *smem, int warp, int units) {
    unsigned char *p = smem + size_t(warp) * back_bytes(units);
    WarpHeadsBack h;
    h.x = reinterpret_cast<float4 *>(p);
    h.g = reinterpret_cast<float4 *>(p + kStage);
    h.unit = reinterpret_cast<Unit *>(p + 2 * kStage);
    h.inv = reinterpret_cast<float *>(h.unit + units);
    h.mean = h.inv + units;
    return h;
}

// Chunk c of heads from, from + step, .. into shared memory, dy turned back; N heads'
// loads in flight.  PAIR: chunk c + turned with it, its partner in a rotation of halves.
constexpr int kBatch = 4;
template <int TY, int N, bool PAIR>
__device__ __forceinline__ void load_heads(const HeadArgs &a, const WarpHeadsBack &h, int here, int from, int step, int c,
                                           int turned, Turn &kept) {
    constexpr int P = PAIR ? 2 : 1;
    const int runs = a.runs.d;
    for (int u0 = from; u0 < here; u0 += N * step) {
        float4 x[N][P], g[N][P];
        int pos[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = u0 + i * step;
            pos[i] = u < here ? h.unit[u].pos : -1;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                x[i][p] = g[i][p] = make_float4(0, 0, 0, 0);
                if (pos[i] != -1) {
                    g[i][p] = load_four<TY>(a, a.dy, h.unit[u].dy + 4 * (c + p * turned));
                    x[i][p] = load_four<TY>(a, a.x, h.unit[u].x + 4 * (c + p * turned));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = u0 + i * step;
            if (pos[i] != -1) {
                if constexpr (PAIR) rotate_halves<true>(a, kept, pos[i], 4 * c, g[i][0], g[i][P - 1]);
                else if (!a.halves) rotate_adjacent<true>(a, kept, pos[i], c, g[i][0]);
            }
            if (u < here) {
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const int at = chunk_at(u * runs, c + p * turned);
                    h.x[at] = x[i][p];
                    h.g[at] = g[i][p];
                }
            }
        }
    }
}

template <int TY, bool VEC>
__global__ void __launch_bounds__(512) head_backward_kernel(const HeadArgs a, int64_t q_runs) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, runs = a.runs.d;
    const WarpHeadsBack h = back_heads(smem, warp, a.units);
    float *fx = reinterpret_cast<float *>(h.x), *fg = reinterpret_cast<float *>(h.g);
    const int key = blockIdx.x >= q_runs;
    const int64_t run = blockIdx.x - (key ? q_runs : 0);
    const int per_row = key ? a.k : a.q;
    const int64_t total = a.rows * per_row, u0 = run * RUN;
    const int in_run = int(imin64(RUN, total - u0));
    const int here = max(0, min(a.units, in_run - warp * a.units));
    if (lane < here) {
        const int64_t at = u0 + warp * a.units + lane, row = row_of(at, per_row);
        place(a, h.unit[lane], row, int(at - row * per_row) + (key ? a.q : 0));
        h.unit[lane].pos = position_of(a, row);
    }
    __syncwarp();
    const float *gain = key ? a.k_gain : a.q_gain;
    const int turned = a.halves ? a.pairs / 4 : 0;
    if constexpr (VEC) {
        const int sub = lane & ((1 << a.per_shift) - 1), from = lane >> a.per_shift, step = 32 >> a.per_shift;
        for (int w = sub; w < a.per; w += 1 << a.per_shift) {
            Turn kept;
            if (w < turned) load_heads<TY, kBatch / 2, true>(a, h, here, from, step, w, turned, kept);
            else load_heads<TY, kBatch, false>(a, h, here, from, step, w + turned, turned, kept);
        }
    } else {
        each_part<Nothing, 1>(here, a.per, a.per_shift, [&](int u, int j, Nothing &) {
            const Unit t = h.unit[u];
            float g = 0.0f, x = 0.0f;
            if (t.pos != -1) {
                x = load_one<TY>(a, a.x, t.x + j);
                g = rotate_one<true>(a, t.pos, j, [&](int c) { return load_one<TY>(a, a.dy, t.dy + c); });
            }
            fx[value_at(u * runs, j)] = x;
            fg[value_at(u * runs, j)] = g;
        });
    }
    __syncwarp();
    const int first = run_first(a), length = min(RUN, a.dim - first), mine = quotient(lane, a.runs);
    const bool folds = lane < here * runs;
    float acc = 0.0f;
    if (folds) acc = fold_squares<VEC>(a, h.x, lane, length);
    float inv = inv_rms(fold_head(a, acc), float(a.dim), a.eps);
    if (folds && h.unit[mine].pos == -1) inv = 0.0f;             // a row left alone adds +0, whatever eps
    if (folds) {
        auto term = [&](float x, float g, float w) { return __fmul_rn(__fmul_rn(g, w), __fmul_rn(x, inv)); };
        auto chunk = [&](int c) {
            const float4 x = h.x[stage_slot(lane, c)], g = h.g[stage_slot(lane, c)];
            const float4 w = load_const(a, reinterpret_cast<const float4 *>(gain + first) + c);
            acc = c == 0 ? term(x.x, g.x, w.x) : __fadd_rn(acc, term(x.x, g.x, w.x));
            acc = __fadd_rn(acc, term(x.y, g.y, w.y));
            acc = __fadd_rn(acc, term(x.z, g.z, w.z));
            acc = __fadd_rn(acc, term(x.w, g.w, w.w));
        };
        if (VEC && a.dim % RUN == 0) {
#pragma unroll
            for (int c = 0; c < 8; ++c) chunk(c);
        } else if (VEC) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (4 * c < length) chunk(c);
        } else {
            for (int i = 0; i < length; ++i) {
                const int at = 4 * stage_slot(lane, i >> 2) + (i & 3);
                const float t = term(fx[at], fg[at], load_const(a, gain + first + i));
                acc = i == 0 ? t : __fadd_rn(acc, t);
            }
        }
    }
    const float mean = __fdiv_rn(fold_head(a, acc), float(a.dim));
    if (first == 0 && mine < a.units) {
        h.inv[mine] = inv;
        h.mean[mine] = mean;
    }
    __syncwarp();
    auto grad = [&](float x, float g, float w, float iv, float m, float &term) {
        const float xh = __fmul_rn(x, iv);
        term = __fmul_rn(g, xh);
        return __fmul_rn(iv, __fsub_rn(__fmul_rn(g, w), __fmul_rn(xh, m)));
    };
    struct Kept {
        bool there = false;
        float4 w;
    };
    each_part<Kept, 2>(here, a.whole, a.whole_shift, [&](int u, int c, Kept &k) {
        const float iv = h.inv[u], mu = h.mean[u];
        const bool live = h.unit[u].pos != -1;
        if constexpr (VEC) {
            const int at = chunk_at(u * runs, c);
            if (!k.there) k.w = load_const(a, reinterpret_cast<const float4 *>(gain) + c);
            k.there = true;
            const float4 x = h.x[at], g = h.g[at], w = k.w;
            float4 d, t;
            d.x = grad(x.x, g.x, w.x, iv, mu, t.x);
            d.y = grad(x.y, g.y, w.y, iv, mu, t.y);
            d.z = grad(x.z, g.z, w.z, iv, mu, t.z);
            d.w = grad(x.w, g.w, w.w, iv, mu, t.w);
            h.g[at] = t;
            if (live) store_four<TY>(a, a.y, h.unit[u].y + 4 * c, d);
        } else {
            const int at = value_at(u * runs, c);
            float t;
            const float d = grad(fx[at], fg[at], load_const(a, gain + c), iv, mu, t);
            fg[at] = t;
            if (live) store_one<TY>(a, a.y, h.unit[u].y + c, d);
        }
    });
    __syncthreads();
    for (int j = threadIdx.x; j < a.dim; j += blockDim.x) {
        const int chunk = j >> 2;
        float sum = 0.0f;
        for (int w = 0, done = 0; done < in_run; ++w) {
            const float *g = reinterpret_cast<const float *>(back_heads(smem, w, a.units).g) + (j & 3);
            const int of = min(a.units, in_run - done);
#pragma unroll 4
            for (int u = 0; u < of; ++u) {
                const float v = g[4 * chunk_at(u * runs, chunk)];
                sum = done + u == 0 ? v : __fadd_rn(sum, v);
            }
            done += of;
        }
        store_global(a, a.part[key] + run * a.dim + j, sum);
    }
}

// The last levels of the gains' sums: 8 columns a CTA, a thread for each group of 32 run
// results (up to 1024 groups), then two levels in shared memory.
struct GainFold : DbgAccess {
    const float *in[2];
    float *out[2];
    int runs[2];
    int dim;
};
__global__ void __launch_bounds__(1024) gain_fold_kernel(const GainFold a) {
    __shared__ float part[RUN * RUN][9];
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3, set = blockIdx.y, c = blockIdx.x * 8 + tx;
    int n = a.runs[set];
    grid_wait();
    if (n == 0) return;
    int groups = (n + RUN - 1) / RUN;
    if (c < a.dim) {
        for (int g = ty; g < groups; g += 128) {
            const float *in = a.in[set] + int64_t(g) * RUN * a.dim + c;
            const int m = min(RUN, n - g * RUN);
            float v[RUN];
#pragma unroll
            for (int i = 0; i < RUN; ++i)
                if (i < m) v[i] = load_global(a, in + int64_t(i) * a.dim);
            float acc = v[0];
#pragma unroll
            for (int i = 1; i < RUN; ++i)
                if (i < m) acc = __fadd_rn(acc, v[i]);
            part[g][tx] = acc;
        }
    }
    while (groups > 1) {
        __syncthreads();
        n = groups;
        groups = (n + RUN - 1) / RUN;
        float acc = 0.0f;
        if (ty < groups) {
            acc = part[ty * RUN][tx];
            const int m = min(RUN, n - ty * RUN);
#pragma unroll 8
            for (int i = 1; i < m; ++i) acc = __fadd_rn(acc, part[ty * RUN + i][tx]);
        }
        __syncthreads();
        if (ty < groups) part[ty][tx] = acc;
    }
    __syncthreads();
    if (ty == 0 && c < a.dim) store_global(a, a.out[set] + c, part[0][tx]);
}

// ------------------------------------------------------------------- host ----

constexpr int64_t kMostFolded = RUN * RUN * RUN;     // run results the last fold takes

template <int TY, bool VEC, bool NORM, bool BACK>
int launch_forward(const HeadArgs &a, cudaStream_t s) {
    const int64_t blocks = ceil_div(a.rows * (a.q + a.k), int64_t(a.units) * kWarps);
    if (blocks > INT32_MAX) return REPOPS_ERR_UNSUPPORTED;
    head_forward_kernel<TY, VEC, NORM, BACK><<<unsigned(blocks), kWarps * 32, 0, s>>>(a);
    return check_launch();
}

template <int TY>
int forward_typed(const HeadArgs &a, bool vec, cudaStream_t s) {
    if (a.q_gain) return vec ? launch_forward<TY, true, true, false>(a, s) : launch_forward<TY, false, true, false>(a, s);
    if (a.inverse) return vec ? launch_forward<TY, true, false, true>(a, s) : launch_forward<TY, false, false, true>(a, s);
    return vec ? launch_forward<TY, true, false, false>(a, s) : launch_forward<TY, false, false, false>(a, s);
}

// How a warp's lanes share its heads.
void share(HeadArgs &a, bool vec) {
    auto lanes = [](int n) {
        int s = 0;
        while (s < 5 && (1 << s) < n) ++s;
        return s;
    };
    a.runs = divisor(ceil_div(a.dim, RUN));
    a.units = RUN / a.runs.d;
    a.whole = vec ? a.dim / 4 : a.dim;
    a.per = vec && a.halves ? a.dim / 4 - a.pairs / 4 : a.whole;
    a.whole_shift = lanes(a.whole);
    a.per_shift = lanes(a.per);
}

int forward_any(HeadArgs a, int type, bool vec, cudaStream_t s) {
    DeviceInfo di;
    if (const int rc = current_device_info(&di); rc != REPOPS_OK) return rc;
    share(a, vec);
    // fewer heads a warp where a CTA for every SM needs it (one row of 40 heads: 6.2 us
    // against 8.5 with all 16 in a warp)
    while (a.units > 1 && a.rows * (a.q + a.k) < int64_t(a.units) * kWarps * di.sms) a.units = (a.units + 1) / 2;
    switch (type) {
        case REPOPS_TYPE_F32: return forward_typed<REPOPS_TYPE_F32>(a, vec, s);
        case REPOPS_TYPE_F16: return forward_typed<REPOPS_TYPE_F16>(a, vec, s);
        default: return forward_typed<REPOPS_TYPE_BF16>(a, vec, s);
    }
}

template <int TY, bool VEC>
int launch_backward(HeadArgs a, int64_t q_runs, int64_t k_runs, cudaStream_t s) {
    share(a, VEC);
    const int warps = (RUN + a.units - 1) / a.units;
    a.units = (RUN + warps - 1) / warps;             // as many heads for each: 8, not 10 and 2
    const size_t smem = size_t(warps) * back_bytes(a.units);
    auto kern = head_backward_kernel<TY, VEC>;
    if (smem > 48 * 1024)
        if (const int rc = allow_shared(kern, kMostBack); rc != REPOPS_OK) return rc;
    kern<<<unsigned(q_runs + k_runs), unsigned(warps * 32), smem, s>>>(a, q_runs);
    return check_launch();
}

// Run results of the further levels of a gain's sum where there are more than the last
// fold takes (a 32nd of them, and so on).
int64_t level_rows(int64_t runs) { return runs > kMostFolded ? 2 * ceil_div(runs, RUN) + 8 : 0; }

// The checks both directions share; what they return is REPOPS_OK with sizes of
// nothing to do (rows or heads of 0), which the callers look at first.
int check_shape(int64_t rows, int64_t q, int64_t k, int64_t dim, int type) {
    if (rows < 0 || q < 0 || k < 0 || dim < 1 || !known_storage(type)) return REPOPS_ERR_INVALID_ARG;
    if (dim > kMostDim || q > 65536 || k > 65536 || rows > (int64_t(1) << 40)) return REPOPS_ERR_UNSUPPORTED;
    return REPOPS_OK;
}

int check_table(const HeadArgs &a, int64_t rows) {
    if (a.pairs < 0 || 2 * int64_t(a.pairs) > a.dim || (a.pos_wide != 0 && a.pos_wide != 1)) return REPOPS_ERR_INVALID_ARG;
    if (misaligned(a.q_gain, 4) || misaligned(a.k_gain, 4) || misaligned(a.pos, a.pos_wide ? 8 : 4) ||
        (a.pairs && (misaligned(a.cosv, 4) || misaligned(a.sinv, 4))))
        return REPOPS_ERR_INVALID_ARG;
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
    if (!x || !y || misaligned(x, size) || misaligned(y, size)) return REPOPS_ERR_INVALID_ARG;
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
    if (!x || !dy || !dx || misaligned(x, size) || misaligned(dy, size) || misaligned(dx, size) || misaligned(dq_gain, 4) ||
        misaligned(dk_gain, 4))
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
    GainFold f{a};
    f.dim = int(dim);
    float *level = a.part[1] + k_runs * dim;
    auto add = [&](int set, const float *in, float *out, int64_t n) {
        while (rc == REPOPS_OK && n > kMostFolded) {
            const int64_t up = ceil_div(n, RUN);
            const dim3 grid(unsigned(ceil_div(dim, 256)), unsigned(std::min<int64_t>(up, 65535)));
            colsum_pass_kernel<<<grid, 256, 0, stream>>>(n, dim, in, dim, level, dim, a);
            rc = check_launch();
            in = level;
            level += up * dim;
            n = up;
        }
        f.in[set] = in;
        f.out[set] = out;
        f.runs[set] = int(n);
    };
    add(0, a.part[0], dq_gain, q_runs);
    add(1, a.part[1], dk_gain, k_runs);
    if (rc == REPOPS_OK)
        rc = launch_behind(gain_fold_kernel, dim3(unsigned(ceil_div(dim, 8)), 2), 1024, 0, stream, f);
    return w.release(rc);
}
