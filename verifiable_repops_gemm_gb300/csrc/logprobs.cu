// logprobs.cu -- log probabilities of given tokens with their row's entropy, log of
// the sum of exponentials and most likely alternatives, and the gradient of the
// logits: the loss of a language model's step, and what an answer is checked by.
//
// Each step one binary32 rounding unless it says binary64.  c = fl(log2(e) / T):
//   e(x; m): t = max(fl(fl(x - m) * c), -127), k = rint(t), f = t - k (exact),
//            p = 1 + f * q(f) by Horner's rule (q of degree 4 fitted to 2^f on
//            [-1/2, 1/2], relative error 9.2e-8), e = p * 2^k (k = -127: +0)
// A row is cut into segments of 1024 columns, whatever computes them.  A segment's
// m is its own maximum (a NaN wins; 0 stands in for -infinity), so that one pass
// over memory does; its s = sum of e and q = sum of fl(e * t) are folded by column:
// the (up to four) columns of one residue modulo 256 in their order from +0, then
// residues r and r + 128, r + 64, ... r + 1.  (A sum of residues r and r + 2^i is
// one of a coset, so the lanes may hold the residues rotated: rows off a 16-byte
// boundary take the same aligned loads.)  The row, in binary64: M = max m,
// w = e(m; M), S = sum of w * s and Q = sum of w * (q + t(m; M) * s), segments of
// one residue modulo 32 in order, then the residues as above; then
//   lse = M / T + ln S,  logp = (x_t - M) / T - ln S,  H = ln S - ln 2 * Q / S
// with ln S = exponent * ln 2 + 2 z (1 + z^2 / 3 + z^4 / 5 + ...), each rounded once.
//
// Work: 16 binary32 instructions a value for the exponential and both sums (the
// additions of two values issued as one), 1 or 2 for the maximum and widening.
#include <algorithm>
#include <cmath>

#include "fixed_math.cuh"
#include "storage.cuh"

namespace repops {
namespace {

constexpr int kSegment = 1024;       // columns whose sums share a maximum
constexpr int kMostTop = 32;         // alternatives: one a lane
constexpr float kMagic = 12582912.0f;

struct LpArgs : DbgAccess {
    int64_t rows, cols, ld;
    const void *x;
    const int64_t *targets;
    float c;                         // fl(log2(e) / T)
    double inv;                      // 1 / T
    float *logp, *lse, *entropy, *stats;
    int top;
    float *top_logp;
    int64_t *top_ids;
    int segments;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ u64 sub2_rn(u64 a, u64 b) {
    u64 d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// e and t of two values at once.
__device__ __forceinline__ void exp_pair(float x0, float x1, float m, float c, float &e0, float &e1, float &t0, float &t1) {
    float d0, d1, b0, b1, f0, f1;
    unpack2(sub2_rn(pack2(x0, x1), pack2(m, m)), d0, d1);
    t0 = max_nan(__fmul_rn(d0, c), -127.0f);
    t1 = max_nan(__fmul_rn(d1, c), -127.0f);
    const u64 t = pack2(t0, t1), big = add2_rn(t, pack2(kMagic, kMagic));
    unpack2(big, b0, b1);
    unpack2(sub2_rn(t, sub2_rn(big, pack2(kMagic, kMagic))), f0, f1);
    float p0 = 0x1.5bba14p-10f, p1 = 0x1.5bba14p-10f;
    horner2(p0, p1, f0, f1, 0x1.3cea88p-7f);
    horner2(p0, p1, f0, f1, 0x1.c6b752p-5f);
    horner2(p0, p1, f0, f1, 0x1.ebf9bcp-3f);
    horner2(p0, p1, f0, f1, 0x1.62e42ap-1f);
    horner2(p0, p1, f0, f1, 1.0f);
    // the low bits of `big` are k: 2^k with the bits 0 at k = -127
    e0 = __fmul_rn(p0, __uint_as_float((__float_as_uint(b0) << 23) + 0x3f800000u));
    e1 = __fmul_rn(p1, __uint_as_float((__float_as_uint(b1) << 23) + 0x3f800000u));
}

// ------------------------------------------------------------ the segments ----

template <int TY>
struct Lanes {
    static constexpr int N = TY == REPOPS_TYPE_F32 ? 4 : 8;      // values of a 16-byte access
    static constexpr int H = 8 / N;                              // accesses of a lane for 256 columns
};

template <int TY>
__device__ __forceinline__ void load_vector(const DbgAccess &d, const void *p, float *v) {
    if constexpr (TY == REPOPS_TYPE_F32) {
        const float4 w = load_const(d, static_cast<const float4 *>(p));
        v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    } else {
        const uint4 w = load_const(d, static_cast<const uint4 *>(p));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TY == REPOPS_TYPE_BF16) {
                v[2 * i] = __uint_as_float(u[i] << 16);
                v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}

// Column of slot `t` of step `i` of a segment for this lane, `off` columns before
// which the row's first 16-byte boundary lies (lane 0's first `off` slots of a
// step hold the next step's columns: see load_segment).
template <int TY>
__device__ __forceinline__ int slot_col(int i, int t, int off) {
    constexpr int N = Lanes<TY>::N;
    const int lane = threadIdx.x & 31;
    return 256 * (i + (t < off && lane == 0)) + 128 * (t / N) + N * lane + t % N - off;
}

// The 32 values a lane has of the segment that starts at column `base`; those past
// the row's end are -infinity.  off != 0: the row starts `off` values behind a
// 16-byte boundary.
template <int TY, bool SHIFT>
__device__ __forceinline__ void load_segment(const LpArgs &a, const char *row, int off, int64_t base, float (&x)[4][8]) {
    constexpr int N = Lanes<TY>::N, H = Lanes<TY>::H;
    constexpr int size = 16 / N;
    const int lane = threadIdx.x & 31;
    const bool inside = (!SHIFT || base >= off) && base + kSegment + (SHIFT ? N : 0) <= a.cols;
    auto fetch = [&](int i, int h, float *v) {
        const int64_t col = base + 256 * i + 128 * h + N * lane - (SHIFT ? off : 0);
        if (inside || (col >= 0 && col + N <= a.cols)) {
            load_vector<TY>(a, row + col * size, v);
        } else {
#pragma unroll
            for (int t = 0; t < N; ++t)
                v[t] = col + t >= 0 && col + t < a.cols ? load_one<TY>(a, row, col + t) : __int_as_float(0xff800000);
        }
    };
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < H; ++h) fetch(i, h, &x[i][N * h]);
    if constexpr (SHIFT) {
        float last[N];
#pragma unroll
        for (int t = 0; t < N; ++t) last[t] = __int_as_float(0xff800000);
        if (lane == 0 && off != 0) fetch(4, 0, last);
#pragma unroll
        for (int t = 0; t < N; ++t) {
            const bool next = lane == 0 && t < off;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i][t] = next ? (i < 3 ? x[i + 1][t] : last[t]) : x[i][t];
        }
    }
}

// One level of a tree in which this lane's partner is lane ^ MASK: with several
// values a lane each of the two keeps one half of the sums.
template <int MASK, int HAVE>
__device__ __forceinline__ void halve(float (&v)[8]) {
    const bool upper = (threadIdx.x & MASK) != 0;
#pragma unroll
    for (int t = 0; t < HAVE / 2; ++t) {
        const float give = upper ? v[t] : v[t + HAVE / 2], keep = upper ? v[t + HAVE / 2] : v[t];
        v[t] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, MASK));
    }
}
template <int MASK>
__device__ __forceinline__ void pair_up(float (&v)[8]) {
    v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], MASK));
}

// The tree over the 256 residues, 8 a lane.
template <int TY>
__device__ __forceinline__ float fold_residues(float (&v)[8]) {
    if constexpr (TY == REPOPS_TYPE_F32) {
        // residue 128 * (slot / 4) + 4 * lane + slot % 4
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = __fadd_rn(v[t], v[t + 4]);
        halve<16, 4>(v);
        halve<8, 2>(v);
        pair_up<4>(v);
        pair_up<2>(v);
        pair_up<1>(v);
        pair_up<16>(v);              // slots 2 apart, then 1 apart
        pair_up<8>(v);
    } else {
        // residue 8 * lane + slot
        halve<16, 8>(v);
        halve<8, 4>(v);
        halve<4, 2>(v);
        pair_up<2>(v);
        pair_up<1>(v);
        pair_up<16>(v);              // slots 4 apart, 2, 1
        pair_up<8>(v);
        pair_up<4>(v);
    }
    return v[0];
}

__device__ __forceinline__ float warp_max_nan(float m) {
#pragma unroll
    for (int i = 16; i; i >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, i));
    return m;
}

// m, s and q of a segment, the same in every lane.
template <int TY>
__device__ __forceinline__ void segment_sums(const float (&x)[4][8], float c, float &m, float &s, float &q) {
    float a[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) a[t] = max_nan(max_nan(x[0][t], x[1][t]), max_nan(x[2][t], x[3][t]));
#pragma unroll
    for (int n = 4; n; n >>= 1)
#pragma unroll
        for (int t = 0; t < n; ++t) a[t] = max_nan(a[t], a[t + n]);
    m = warp_max_nan(a[0]);
    const float ref = m == __int_as_float(0xff800000) ? 0.0f : m;
    float sv[8], qv[8];
#pragma unroll
    for (int t = 0; t < 8; t += 2) {
        u64 ss = pack2(0.0f, 0.0f), qq = pack2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float e0, e1, t0, t1;
            exp_pair(x[i][t], x[i][t + 1], ref, c, e0, e1, t0, t1);
            ss = add2_rn(ss, pack2(e0, e1));
            qq = add2_rn(qq, pack2(__fmul_rn(e0, t0), __fmul_rn(e1, t1)));
        }
        unpack2(ss, sv[t], sv[t + 1]);
        unpack2(qq, qv[t], qv[t + 1]);
    }
    s = fold_residues<TY>(sv);
    q = fold_residues<TY>(qv);
}

// ------------------------------------------------------------ alternatives ----

// Whole numbers in the order of the values, NaN above all and both zeros the same;
// the lower column first among equals.  Never 0.
__device__ __forceinline__ u64 order_key(float v, uint32_t col) {
    uint32_t b = v == 0.0f ? 0u : __float_as_uint(v);
    b = v != v ? 0xffffffffu : ((b >> 31) ? ~b : b | 0x80000000u);
    return (u64(b) << 32) | (0xffffffffu - col);
}
__device__ __forceinline__ float key_value(u64 k) {
    const uint32_t b = uint32_t(k >> 32);
    return __uint_as_float((b >> 31) ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ uint32_t key_col(u64 k) { return 0xffffffffu - uint32_t(k); }

// A warp's list of the n largest keys, lane i's the i-th.
struct TopList {
    u64 mine = 0, least = 0;         // least: the n-th key
    // Takes in one key of each lane (0: none).
    __device__ __forceinline__ void add(u64 cand, int n) {
        const int lane = threadIdx.x & 31;
        uint32_t left = __ballot_sync(0xffffffffu, cand > least);
        while (left) {
            const u64 k = __shfl_sync(0xffffffffu, cand, __ffs(left) - 1);
            left &= left - 1;
            if (k <= least) continue;
            const int at = __popc(__ballot_sync(0xffffffffu, mine > k));
            const u64 above = __shfl_up_sync(0xffffffffu, mine, 1);
            if (lane == at) mine = k;
            else if (lane > at) mine = above;
            least = __shfl_sync(0xffffffffu, mine, n - 1);
        }
    }
};

// --------------------------------------------------------------- the row ----

constexpr double kLn2 = 0x1.62e42fefa39efp-1;

// ln of a finite S >= 1/2, of 0, or of a NaN.
__device__ double ln_fixed(double S) {
    if (!(S > 0.0)) return S == 0.0 ? __longlong_as_double(0xfff0000000000000ll) : S;
    const long long bits = __double_as_longlong(S);
    int e = int((bits >> 52) & 0x7ff) - 1023;
    double f = __longlong_as_double((bits & 0xfffffffffffffll) | 0x3ff0000000000000ll);
    if (e == 1024) return S;
    if (f > 1.41421356237309504880) {
        f = __dmul_rn(f, 0.5);
        ++e;
    }
    const double z = __ddiv_rn(__dadd_rn(f, -1.0), __dadd_rn(f, 1.0)), zz = __dmul_rn(z, z);
    double p = 1.0 / 23.0;
#pragma unroll
    for (int n = 10; n >= 0; --n) p = __dadd_rn(__dmul_rn(p, zz), 1.0 / (2 * n + 1));
    return __dadd_rn(__dmul_rn(double(e), kLn2), __dmul_rn(__dmul_rn(2.0, z), p));
}

__device__ __forceinline__ double shift_of(float x, float M, double inv) {
    return __dmul_rn(__dadd_rn(double(x), -double(M)), inv);
}
__device__ __forceinline__ float logp_of(float x, float M, double inv, double lnS) {
    if (x == __int_as_float(0xff800000) && M < __int_as_float(0x7f800000)) return x;     // impossible, also where all is
    return __double2float_rn(__dadd_rn(shift_of(x, M, inv), -lnS));
}

// Shared memory of a row's first CTA: m, s and q of the segments, then each warp's keys.
__host__ __device__ inline size_t lp_smem(int segments, int warps, int top) {
    const size_t sums = (size_t(segments) * 12 + 15) / 16 * 16;
    return sums + (top ? size_t(warps + 1) * kMostTop * sizeof(u64) : 0) + 16;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Into the shared memory of the cluster's first CTA.
__device__ __forceinline__ void store_first(float *p, float v) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_addr(p)));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// A cluster a row; its warps take the segments in turn.
template <int TY, bool SHIFT>
__global__ void __launch_bounds__(256) logprobs_kernel(const LpArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    float *sm = reinterpret_cast<float *>(smem), *ss = sm + a.segments, *sq = ss + a.segments;
    u64 *keys = reinterpret_cast<u64 *>(smem + (size_t(a.segments) * 12 + 15) / 16 * 16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const uint32_t ctas = cluster_size(), rank = cluster_rank();
    if (!REPOPS_DBG_SMEM_OK(lp_smem(a.segments, warps, a.top), a.status)) return;
    const int64_t row = blockIdx.x / ctas;
    constexpr int size = TY == REPOPS_TYPE_F32 ? 4 : 2;
    const char *x = static_cast<const char *>(a.x) + row * a.ld * size;
    const int off = SHIFT ? int(reinterpret_cast<uintptr_t>(x) % 16) / size : 0;
    float v[4][8];
    if (ctas > 1) cluster_arrive();
    bool started = ctas == 1;
    for (int j = int(rank) * warps + warp; j < a.segments; j += int(ctas) * warps) {
        load_segment<TY, SHIFT>(a, x, off, int64_t(j) * kSegment, v);
        float m, s, q;
        segment_sums<TY>(v, a.c, m, s, q);
        if (!started) {              // the first CTA's shared memory is there
            cluster_wait();
            started = true;
        }
        if (lane == 0) {
            if (ctas > 1) {
                store_first(sm + j, m);
                store_first(ss + j, s);
                store_first(sq + j, q);
            } else {
                sm[j] = m;
                ss[j] = s;
                sq[j] = q;
            }
        }
    }
    if (ctas > 1) {
        if (!started) cluster_wait();
        cluster_arrive();
        if (rank != 0) {
            cluster_wait();
            return;
        }
        cluster_wait();
    } else {
        __syncthreads();
    }
    // the alternatives are in the `top` segments with the largest maxima (the first
    // among equals): any other segment has that many values in front of its own
    if (a.top && warp == (warps > 1 ? 1 : 0)) {
        TopList best;
        for (int j = lane; j - lane < a.segments; j += 32)
            best.add(j < a.segments ? order_key(sm[j], uint32_t(j)) : 0, a.top);
        keys[warps * kMostTop + lane] = best.mine;
    }
    float M = __int_as_float(0xff800000);
    double S = 0.0, Q = 0.0, lnS = 0.0;
    if (warp == 0) {
        for (int j = lane; j < a.segments; j += 32) M = max_nan(M, sm[j]);
        M = warp_max_nan(M);
        const float ref = M == __int_as_float(0xff800000) ? 0.0f : M;
        for (int j = lane; j < a.segments; j += 32) {
            float e, e1, t, t1;
            exp_pair(sm[j], sm[j], ref, a.c, e, e1, t, t1);
            S = __dadd_rn(S, __dmul_rn(double(e), double(ss[j])));
            Q = __dadd_rn(Q, __dmul_rn(double(e), __dadd_rn(double(sq[j]), __dmul_rn(double(t), double(ss[j])))));
        }
#pragma unroll
        for (int i = 16; i; i >>= 1) {
            S = __dadd_rn(S, __shfl_xor_sync(0xffffffffu, S, i));
            Q = __dadd_rn(Q, __shfl_xor_sync(0xffffffffu, Q, i));
        }
        lnS = ln_fixed(S);
        if (lane == 0) {
            const bool empty = S == 0.0;
            const int64_t t = a.targets ? load_const(a, a.targets + row) : -1;
            float lp = 0.0f;
            if (t >= a.cols) lp = __int_as_float(0x7fffffff);
            else if (t >= 0) lp = logp_of(load_one<TY>(a, x, t), M, a.inv, lnS);
            const float H = empty ? 0.0f : __double2float_rn(__dadd_rn(lnS, -__dmul_rn(kLn2, __ddiv_rn(Q, S))));
            store_global(a, a.logp + row, lp);
            store_global(a, a.lse + row, empty ? M : __double2float_rn(__dadd_rn(__dmul_rn(double(M), a.inv), lnS)));
            store_global(a, a.entropy + row, H);
            store_global(a, reinterpret_cast<float4 *>(a.stats) + row,
                         make_float4(M, empty ? 0.0f : __double2float_rn(__ddiv_rn(1.0, S)), __double2float_rn(lnS), H));
        }
    }
    if (!a.top) return;
    __syncthreads();
    {
        TopList best;
        const int chosen = min(a.top, a.segments);
        for (int n = warp; n < chosen; n += warps) {
            const uint32_t j = key_col(keys[warps * kMostTop + n]);
            load_segment<TY, SHIFT>(a, x, off, int64_t(j) * kSegment, v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const int64_t col = int64_t(j) * kSegment + slot_col<TY>(i, t, off);
                    best.add(col < a.cols ? order_key(v[i][t], uint32_t(col)) : 0, a.top);
                }
        }
        keys[warp * kMostTop + lane] = best.mine;
    }
    __syncthreads();
    if (warp == 0) {
        TopList best;
        for (int w = 0; w < warps; ++w) best.add(keys[w * kMostTop + lane], a.top);
        if (lane < a.top) {
            store_global(a, a.top_ids + row * a.top + lane, int64_t(key_col(best.mine)));
            store_global(a, a.top_logp + row * a.top + lane, logp_of(key_value(best.mine), M, a.inv, lnS));
        }
    }
}

// ---------------------------------------------------------------- gradient ----

struct LpGradArgs : DbgAccess {
    int64_t rows, cols, ld, ldd;
    const void *x;
    void *dx;
    const int64_t *targets;
    const float *stats, *dlogp, *dentropy;
    float c, inv;
};

// dx = fl(p * fl(A + fl(B * t))), p = fl(e * (1/S)); at the target + G.  One or two
// 16-byte accesses a thread.
template <int TY, bool ENTROPY, bool VEC>
__global__ void __launch_bounds__(256) logprobs_backward_kernel(const LpGradArgs a) {
    constexpr int N = VEC ? Lanes<TY>::N : 8;
    constexpr int size = TY == REPOPS_TYPE_F32 ? 4 : 2;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float4 st = load_const(a, reinterpret_cast<const float4 *>(a.stats) + row);
        const int64_t target = a.targets ? load_const(a, a.targets + row) : -1;
        float w = target >= 0 && a.dlogp ? load_const(a, a.dlogp + row) : 0.0f;
        if (target >= a.cols && a.dlogp) w = __int_as_float(0x7fffffff);
        const float h = ENTROPY ? load_const(a, a.dentropy + row) : 0.0f;
        const bool empty = st.x == __int_as_float(0xff800000);
        const float ref = empty ? 0.0f : st.x;
        float A = w, B = 0.0f;
        if (ENTROPY) {
            A = __fadd_rn(A, __fmul_rn(h, __fsub_rn(st.w, st.z)));
            B = -__fmul_rn(__fmul_rn(a.inv, 0x1.62e430p-1f), h);
        }
        A = empty ? 0.0f : -__fmul_rn(a.inv, A);
        if (empty) B = 0.0f;
        const float G = empty ? 0.0f : __fmul_rn(a.inv, w);
        const char *x = static_cast<const char *>(a.x) + row * a.ld * size;
        char *dx = static_cast<char *>(a.dx) + row * a.ldd * size;
        const int off = VEC ? int(reinterpret_cast<uintptr_t>(x) % 16) / size : 0;
        const int64_t first = (blockIdx.x * int64_t(blockDim.x) + threadIdx.x) * N - off;
        const int64_t step = int64_t(gridDim.x) * blockDim.x * N;
        for (int64_t col = first; col < a.cols; col += step) {
            float v[8];
            const bool whole = VEC && col >= 0 && col + N <= a.cols;
            if (whole) {
                load_vector<TY>(a, x + col * size, v);
            } else {
#pragma unroll
                for (int t = 0; t < N; ++t)
                    v[t] = col + t >= 0 && col + t < a.cols ? load_one<TY>(a, x, col + t) : 0.0f;
            }
#pragma unroll
            for (int t = 0; t < N; t += 2) {
                float e0, e1, t0, t1;
                exp_pair(v[t], v[t + 1], ref, a.c, e0, e1, t0, t1);
                const float p0 = __fmul_rn(e0, st.y), p1 = __fmul_rn(e1, st.y);
                v[t] = __fmul_rn(p0, ENTROPY ? __fadd_rn(A, __fmul_rn(B, t0)) : A);
                v[t + 1] = __fmul_rn(p1, ENTROPY ? __fadd_rn(A, __fmul_rn(B, t1)) : A);
            }
            const int64_t at = target - col;
            if (at >= 0 && at < N) {
#pragma unroll
                for (int t = 0; t < N; ++t)
                    if (t == at) v[t] = __fadd_rn(v[t], G);
            }
            if (whole) {
                if constexpr (TY == REPOPS_TYPE_F32) {
                    store_once(a, reinterpret_cast<float4 *>(dx + col * size), make_float4(v[0], v[1], v[2], v[3]));
                } else {
                    uint4 u;
                    u.x = narrowed<TY>(v[0]) | (narrowed<TY>(v[1]) << 16);
                    u.y = narrowed<TY>(v[2]) | (narrowed<TY>(v[3]) << 16);
                    u.z = narrowed<TY>(v[4]) | (narrowed<TY>(v[5]) << 16);
                    u.w = narrowed<TY>(v[6]) | (narrowed<TY>(v[7]) << 16);
                    store_once(a, reinterpret_cast<uint4 *>(dx + col * size), u);
                }
            } else {
#pragma unroll
                for (int t = 0; t < N; ++t)
                    if (col + t >= 0 && col + t < a.cols) store_one<TY>(a, dx, col + t, v[t]);
            }
        }
    }
}

// ------------------------------------------------------------------- host ----

template <int TY, bool SHIFT>
int launch_logprobs(const LpArgs &a, cudaStream_t s) {
    DeviceInfo di;
    if (const int rc = current_device_info(&di); rc != REPOPS_OK) return rc;
    int warps = 1;
    while (warps < 8 && warps < a.segments) warps *= 2;
    // few rows: a row's segments are shared by the CTAs of a cluster
    unsigned ctas = 1;
    while (ctas < 8 && a.rows * ctas < 2 * di.sms && int(2 * ctas) * warps <= a.segments) ctas *= 2;
    const size_t smem = lp_smem(a.segments, warps, a.top);
    auto kern = logprobs_kernel<TY, SHIFT>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return set_cuda_error(e);
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.rows * ctas));
    cfg.blockDim = dim3(unsigned(warps * 32));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    return e == cudaSuccess ? REPOPS_OK : set_cuda_error(e);
}

template <int TY>
int launch_backward(const LpGradArgs &a, bool vec, cudaStream_t s) {
    const int n = vec ? Lanes<TY>::N : 8;
    const int64_t blocks = (a.cols + (vec ? n : 0) + 256 * n - 1) / (256 * n);
    const dim3 grid(unsigned(std::min<int64_t>(blocks, 1 << 20)), unsigned(std::min<int64_t>(a.rows, 65535)));
    if (a.dentropy) {
        if (vec) logprobs_backward_kernel<TY, true, true><<<grid, 256, 0, s>>>(a);
        else logprobs_backward_kernel<TY, true, false><<<grid, 256, 0, s>>>(a);
    } else {
        if (vec) logprobs_backward_kernel<TY, false, true><<<grid, 256, 0, s>>>(a);
        else logprobs_backward_kernel<TY, false, false><<<grid, 256, 0, s>>>(a);
    }
    return check_launch();
}

constexpr int64_t kMostColumns = int64_t(16000) * kSegment;      // 187.5 KB of sums
constexpr double kLog2e = 0x1.71547652b82fep+0;

bool good_temperature(float t) { return t >= 1e-6f && t <= 1e6f; }

}  // namespace
}  // namespace repops

using namespace repops;

extern "C" int repops_token_logprobs(int64_t rows, int64_t cols, const void *x, int x_type, int64_t ldx,
                                     const int64_t *targets, float temperature, int top, float *logp, float *lse,
                                     float *entropy, float *stats, float *top_logp, int64_t *top_ids,
                                     cudaStream_t stream) {
    if (rows < 0 || cols < 1 || !known_storage(x_type) || !good_temperature(temperature) || top < 0 || top > cols)
        return REPOPS_ERR_INVALID_ARG;
    if (cols > kMostColumns || top > kMostTop || rows > (int64_t(1) << 27)) return REPOPS_ERR_UNSUPPORTED;
    if (rows == 0) return REPOPS_OK;
    uint64_t xb;
    if (!x || !logp || !lse || !entropy || !stats || (top && (!top_logp || !top_ids)) ||
        reinterpret_cast<uintptr_t>(stats) % 16 != 0 || reinterpret_cast<uintptr_t>(x) % storage_size(x_type) != 0 ||
        !span_bytes(rows, cols, ldx, storage_size(x_type), &xb))
        return REPOPS_ERR_INVALID_ARG;
    const uint64_t vb = uint64_t(rows) * 4u, tb = uint64_t(rows) * uint64_t(top);
    const struct { void *p; uint64_t b; } outs[6] = {{logp, vb}, {lse, vb}, {entropy, vb}, {stats, 4 * vb},
                                                     {top ? top_logp : nullptr, 4 * tb}, {top ? top_ids : nullptr, 8 * tb}};
    for (int i = 0; i < 6; ++i) {
        if (!outs[i].p) continue;
        if (ranges_overlap(outs[i].p, outs[i].b, x, xb) ||
            (targets && ranges_overlap(outs[i].p, outs[i].b, targets, uint64_t(rows) * 8u)))
            return REPOPS_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (outs[j].p && ranges_overlap(outs[i].p, outs[i].b, outs[j].p, outs[j].b)) return REPOPS_ERR_ALIAS;
    }
    LpArgs a{};
    a.rows = rows; a.cols = cols; a.ld = ldx;
    a.x = x;
    a.targets = targets;
    a.c = float(kLog2e / double(temperature));
    a.inv = 1.0 / double(temperature);
    a.logp = logp; a.lse = lse; a.entropy = entropy; a.stats = stats;
    a.top = top; a.top_logp = top_logp; a.top_ids = top_ids;
    a.segments = int((cols + kSegment - 1) / kSegment);
    a.reads(x, xb);
    a.reads(targets, uint64_t(rows) * 8u);
    for (const auto &o : outs) a.writes(o.p, o.b);
    if (const int rc = a.arm(); rc != REPOPS_OK) return rc;
    const bool aligned = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx * storage_size(x_type) % 16 == 0;
    switch (x_type) {
        case REPOPS_TYPE_F32:
            return aligned ? launch_logprobs<REPOPS_TYPE_F32, false>(a, stream) : launch_logprobs<REPOPS_TYPE_F32, true>(a, stream);
        case REPOPS_TYPE_F16:
            return aligned ? launch_logprobs<REPOPS_TYPE_F16, false>(a, stream) : launch_logprobs<REPOPS_TYPE_F16, true>(a, stream);
        default:
            return aligned ? launch_logprobs<REPOPS_TYPE_BF16, false>(a, stream) : launch_logprobs<REPOPS_TYPE_BF16, true>(a, stream);
    }
}

extern "C" int repops_token_logprobs_backward(int64_t rows, int64_t cols, const void *x, int x_type, int64_t ldx,
                                              const int64_t *targets, float temperature, const float *stats,
                                              const float *dlogp, const float *dentropy, void *dx, int64_t lddx,
                                              cudaStream_t stream) {
    if (rows < 0 || cols < 1 || !known_storage(x_type) || !good_temperature(temperature)) return REPOPS_ERR_INVALID_ARG;
    if (cols > kMostColumns || rows > (int64_t(1) << 27)) return REPOPS_ERR_UNSUPPORTED;
    if (rows == 0) return REPOPS_OK;
    const unsigned size = storage_size(x_type);
    uint64_t xb, db;
    if (!x || !dx || !stats || (!dlogp && !dentropy) || (dlogp && !targets) || reinterpret_cast<uintptr_t>(stats) % 16 != 0 ||
        reinterpret_cast<uintptr_t>(x) % size != 0 || reinterpret_cast<uintptr_t>(dx) % size != 0 ||
        !span_bytes(rows, cols, ldx, size, &xb) || !span_bytes(rows, cols, lddx, size, &db))
        return REPOPS_ERR_INVALID_ARG;
    const uint64_t vb = uint64_t(rows) * 4u;
    if (!(dx == x && lddx == ldx) && ranges_overlap(dx, db, x, xb)) return REPOPS_ERR_ALIAS;
    if (ranges_overlap(dx, db, stats, 4 * vb) || (dlogp && ranges_overlap(dx, db, dlogp, vb)) ||
        (dentropy && ranges_overlap(dx, db, dentropy, vb)) || (targets && ranges_overlap(dx, db, targets, 2 * vb)))
        return REPOPS_ERR_ALIAS;
    LpGradArgs a{};
    a.rows = rows; a.cols = cols; a.ld = ldx; a.ldd = lddx;
    a.x = x; a.dx = dx;
    a.targets = targets;
    a.stats = stats; a.dlogp = dlogp; a.dentropy = dentropy;
    a.c = float(kLog2e / double(temperature));
    a.inv = 1.0f / temperature;
    a.reads(x, xb);
    a.reads(targets, 2 * vb);
    a.reads(stats, 4 * vb);
    a.reads(dlogp, vb);
    a.reads(dentropy, vb);
    a.writes(dx, db);
    if (const int rc = a.arm(); rc != REPOPS_OK) return rc;
    // every row of dx as far from a 16-byte boundary as the same row of x
    const bool vec = (reinterpret_cast<uintptr_t>(x) - reinterpret_cast<uintptr_t>(dx)) % 16 == 0 &&
                     (ldx - lddx) * int64_t(size) % 16 == 0;
    switch (x_type) {
        case REPOPS_TYPE_F32: return launch_backward<REPOPS_TYPE_F32>(a, vec, stream);
        case REPOPS_TYPE_F16: return launch_backward<REPOPS_TYPE_F16>(a, vec, stream);
        default: return launch_backward<REPOPS_TYPE_BF16>(a, vec, stream);
    }
}
