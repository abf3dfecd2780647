// logprobs.cu -- log probabilities of given tokens with their row's entropy, log of
// the sum of exponentials and most likely alternatives, and the gradient of the
// logits: the loss of a language model's step, and what an answer is checked by.
//
// Each step one binary32 rounding.  c = fl(log2(e) / T):
//   e(x; m): t = max(fl(fl(x - m) * c), -127), n = rint(32 t), f = t - n / 32 (exact),
//            p = 1 + f * (a + f * b) by Horner's rule (fitted to 2^f on [-1/64, 1/64],
//            relative error 5.3e-8), e = fl(p * 2^(n / 32)), the power with the bits of
//            fl(2^(j / 32)), j = n mod 32, and (n - j) / 32 added to their exponent (so
//            +0 at t = -127)
// A row is cut into segments of 4096 columns and those into blocks of 1024, whatever
// computes them, so that one pass over memory does and a row can be shared.  A
// segment takes its blocks in order with the maximum so far, m (a NaN wins; inside e
// and t 0 stands in for -infinity): where a block raises it from m to m', what has
// been summed is brought along, q = fl(w * fl(q + fl(d * s))), s = fl(w * s), w =
// e(m; m'), d = t(m; m').  s sums e and q fl(e * t), for each residue of the column
// modulo 256 in the columns' order from +0; at the segment's end residues r and r +
// 128, r + 64, ... r + 1 are added.  (A sum of residues r and r + 2^i is one of a
// coset, so the lanes may hold the residues rotated: rows off a 16-byte boundary take
// the same aligned loads.)  The row: M = max m, w = e(m; M), S = sum of w * s and Q =
// sum of w * (q + t(m; M) * s), segments of one residue modulo 32 in order, then the
// residues as above; then
//   lse = M / T + ln S,  logp = (x_t - M) / T - ln S,  H = ln S - ln 2 * Q / S
// with ln S = E ln 2 + 2 z (1 + z^2 / 3 + ... + z^8 / 9), z = (F - 1) / (F + 1), S = F
// * 2^E.  (Binary64 would cost more than the sums of a short row: an SM does two such
// operations a clock.)
//
// The alternatives lie in the `top` blocks with the largest maxima (the first among
// equals): any other block has that many values in front of its own.  Those are read
// again, and of them the values that reach the least of these maxima are ranked by
// counting, which takes few dependent steps; ties by the thousand take lists.
//
#include <algorithm>
#include <cmath>

#include "fixed_math.cuh"
#include "storage.cuh"

namespace repops {
namespace {

constexpr int kBlock = 1024;         // columns a warp holds at once
constexpr int kSegment = 4 * kBlock; // columns whose sums are folded together
constexpr int64_t kMostColumns = int64_t(16000) * kBlock;        // 114 KB of sums and maxima
constexpr int kMostTop = 32;         // alternatives: one a lane
constexpr int kMostListed = 256;     // values ranked by counting
constexpr float kMagic = 393216.0f;   // 1.5 * 2^18: adding it rounds to a 32nd

struct LpArgs : DbgAccess {
    int64_t rows, cols, ld;
    const void *x;
    const int64_t *targets;
    float c;                         // fl(log2(e) / T)
    float inv;                       // fl(1 / T)
    float *logp, *lse, *entropy, *stats;
    int top;
    float *top_logp;
    int64_t *top_ids;
    int segments, blocks;
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

__device__ __forceinline__ u64 mul2_rn(u64 a, u64 b) {
    u64 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// fl(2^(j / 32)) less j << 18: what (n << 18) has of j besides the exponent.  Lane j
// holds the j-th in a register and a shuffle looks it up, which takes the place of
// three more degrees of the polynomial: these kernels are bound by the instructions
// they issue, of which a packed addition is two.
__constant__ uint32_t kPowers[32] = {
#define P(bits, j) (bits) - ((j) << 18)
    P(0x3f800000u, 0u),  P(0x3f82cd87u, 1u),  P(0x3f85aac3u, 2u),  P(0x3f88980fu, 3u),  P(0x3f8b95c2u, 4u),
    P(0x3f8ea43au, 5u),  P(0x3f91c3d3u, 6u),  P(0x3f94f4f0u, 7u),  P(0x3f9837f0u, 8u),  P(0x3f9b8d3au, 9u),
    P(0x3f9ef532u, 10u), P(0x3fa27043u, 11u), P(0x3fa5fed7u, 12u), P(0x3fa9a15bu, 13u), P(0x3fad583fu, 14u),
    P(0x3fb123f6u, 15u), P(0x3fb504f3u, 16u), P(0x3fb8fbafu, 17u), P(0x3fbd08a4u, 18u), P(0x3fc12c4du, 19u),
    P(0x3fc5672au, 20u), P(0x3fc9b9beu, 21u), P(0x3fce248cu, 22u), P(0x3fd2a81eu, 23u), P(0x3fd744fdu, 24u),
    P(0x3fdbfbb8u, 25u), P(0x3fe0ccdfu, 26u), P(0x3fe5b907u, 27u), P(0x3feac0c7u, 28u), P(0x3fefe4bau, 29u),
    P(0x3ff5257du, 30u), P(0x3ffa83b3u, 31u)
#undef P
};

// e and t of two values at once, by whole warps, `power` being the lane's of kPowers.
// The one packed product is followed by a maximum: no addition could be fused with it
// to other bits.
__device__ __forceinline__ void exp_pair(uint32_t power, float x0, float x1, float m, float c, float &e0, float &e1,
                                         float &t0, float &t1) {
    float b0, b1, f0, f1;
    unpack2(mul2_rn(sub2_rn(pack2(x0, x1), pack2(m, m)), pack2(c, c)), t0, t1);
    t0 = max_nan(t0, -127.0f);
    t1 = max_nan(t1, -127.0f);
    const u64 t = pack2(t0, t1), big = add2_rn(t, pack2(kMagic, kMagic));      // its low bits are n
    unpack2(big, b0, b1);
    unpack2(sub2_rn(t, sub2_rn(big, pack2(kMagic, kMagic))), f0, f1);
    const uint32_t n0 = __float_as_uint(b0), n1 = __float_as_uint(b1);
    float p0 = 0x1.ebfbe0p-3f, p1 = 0x1.ebfbe0p-3f;
    horner2(p0, p1, f0, f1, 0x1.62e584p-1f);
    horner2(p0, p1, f0, f1, 1.0f);
    e0 = __fmul_rn(p0, __uint_as_float((n0 << 18) + __shfl_sync(0xffffffffu, power, n0)));
    e1 = __fmul_rn(p1, __uint_as_float((n1 << 18) + __shfl_sync(0xffffffffu, power, n1)));
}

// Whole numbers in the order of the values, NaN above all and both zeros the same.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = v == 0.0f ? 0u : __float_as_uint(v);
    return v != v ? 0xffffffffu : ((b >> 31) ? ~b : b | 0x80000000u);
}

// -------------------------------------------------------------- the blocks ----

template <int TY>
struct Lanes {
    static constexpr int N = TY == REPOPS_TYPE_F32 ? 4 : 8;      // values of a 16-byte access
    static constexpr int H = 8 / N;                              // accesses of a lane for 256 columns
    static constexpr uint32_t kEmpty =                           // -infinity in every value of a word
        TY == REPOPS_TYPE_F32 ? 0xff800000u : TY == REPOPS_TYPE_F16 ? 0xfc00fc00u : 0xff80ff80u;
};

// The 32 values a lane has of a block, as stored: step i (256 columns) is 8 of them,
// slot t of which is column 256 i + 128 * (t / N) + N * lane + t % N of the block.
template <int TY>
struct Raw {
    uint32_t w[4][4 * Lanes<TY>::H];
};

// Values t and t + 1 (t even) of a step.
template <int TY>
__device__ __forceinline__ void two_of(const uint32_t *w, int t, float &a, float &b) {
    if constexpr (TY == REPOPS_TYPE_F32) {
        a = __uint_as_float(w[t]);
        b = __uint_as_float(w[t + 1]);
    } else if constexpr (TY == REPOPS_TYPE_BF16) {
        a = __uint_as_float(w[t / 2] << 16);
        b = __uint_as_float(w[t / 2] & 0xffff0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[t / 2]));
        a = f.x;
        b = f.y;
    }
}

// A row that starts `off` values behind a 16-byte boundary takes its accesses from
// that boundary.  Lane 0's first `off` slots of a step are then the last columns of
// the step before: `mask` has their bits (lane 0's alone), and load_block puts the
// next step's in their place.
template <int TY>
__device__ __forceinline__ void slot_masks(int off, uint32_t (&mask)[4]) {
    const int n = (threadIdx.x & 31) == 0 ? off : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (TY == REPOPS_TYPE_F32) mask[j] = j < n ? 0xffffffffu : 0u;
        else mask[j] = (2 * j < n ? 0xffffu : 0u) | (2 * j + 1 < n ? 0xffff0000u : 0u);
    }
}
template <int TY>
__device__ __forceinline__ int slot_col(int i, int t, int off) {
    constexpr int N = Lanes<TY>::N;
    const int lane = threadIdx.x & 31;
    return 256 * (i + (t < off && lane == 0)) + 128 * (t / N) + N * lane + t % N - off;
}

// The block that starts at column `base`; columns past the row's end are -infinity.
template <int TY, bool SHIFT>
__device__ __forceinline__ void load_block(const LpArgs &a, const char *row, int off, const uint32_t (&mask)[4], int base,
                                           Raw<TY> &r) {
    constexpr int N = Lanes<TY>::N, H = Lanes<TY>::H, size = 16 / N;
    const int lane = threadIdx.x & 31, cols = int(a.cols);
    const char *at = row + int64_t(base + N * lane - (SHIFT ? off : 0)) * size;
    auto fetch = [&](int i, int h, uint32_t *w) {
        const uint4 u = load_const(a, reinterpret_cast<const uint4 *>(at + (256 * i + 128 * h) * size));
        w[0] = u.x;
        w[1] = u.y;
        w[2] = u.z;
        w[3] = u.w;
    };
    auto fetch_edge = [&](int i, int h, uint32_t *w) {       // one of them may leave the row
        const int col = base + 256 * i + 128 * h + N * lane - (SHIFT ? off : 0);
        if (col >= 0 && col + N <= cols) return fetch(i, h, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = Lanes<TY>::kEmpty;
            if constexpr (TY == REPOPS_TYPE_F32) {
                if (col + j >= 0 && col + j < cols) w[j] = load_const(a, reinterpret_cast<const uint32_t *>(row) + col + j);
            } else {
                const uint16_t *p = reinterpret_cast<const uint16_t *>(row);
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (col + 2 * j + s >= 0 && col + 2 * j + s < cols)
                        w[j] = __byte_perm(w[j], load_const(a, p + col + 2 * j + s), s ? 0x5410 : 0x3254);
            }
        }
    };
    const bool inside = (!SHIFT || base >= off) && base + kBlock + (SHIFT ? N : 0) <= cols;
    if (inside) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < H; ++h) fetch(i, h, &r.w[i][4 * h]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < H; ++h) fetch_edge(i, h, &r.w[i][4 * h]);
    }
    if constexpr (SHIFT) {
        uint32_t last[4] = {Lanes<TY>::kEmpty, Lanes<TY>::kEmpty, Lanes<TY>::kEmpty, Lanes<TY>::kEmpty};
        if (lane == 0 && off != 0) fetch_edge(4, 0, last);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) r.w[i][j] = (r.w[i][j] & ~mask[j]) | ((i < 3 ? r.w[i + 1][j] : last[j]) & mask[j]);
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
    float all;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(all) : "f"(m));
    return all;
}

// The largest of a lane's values of a block, and of the block's, the same in every lane.
template <int TY>
__device__ __forceinline__ float lane_max(const Raw<TY> &r) {
    float m;
    if constexpr (TY == REPOPS_TYPE_F32) {
        m = __uint_as_float(r.w[0][0]);
#pragma unroll
        for (int n = 1; n < 31; n += 2)
            asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(__uint_as_float(r.w[n / 8][n % 8])),
                "f"(__uint_as_float(r.w[(n + 1) / 8][(n + 1) % 8])));
        m = max_nan(m, __uint_as_float(r.w[3][7]));
    } else {
        uint32_t u = r.w[0][0];
#pragma unroll
        for (int n = 1; n < 16; ++n) {
            if constexpr (TY == REPOPS_TYPE_F16) asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(u) : "r"(r.w[n / 4][n % 4]));
            else asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(u) : "r"(r.w[n / 4][n % 4]));
        }
        float x, y;
        two_of<TY>(&u, 0, x, y);
        m = max_nan(x, y);
    }
    return m;
}
template <int TY>
__device__ __forceinline__ float block_max(const Raw<TY> &r) {
    return warp_max_nan(lane_max<TY>(r));
}

constexpr float kMinusInf = -__builtin_inff();

// What stands in for a maximum inside e and t.
__device__ __forceinline__ float reference(float m) { return m == kMinusInf ? 0.0f : m; }

// A segment's sums so far, the residues of this lane.
struct Sums {
    float m;
    u64 s[4], q[4];
    __device__ __forceinline__ void clear() {
        m = kMinusInf;
#pragma unroll
        for (int t = 0; t < 4; ++t) s[t] = q[t] = pack2(0.0f, 0.0f);
    }
    // Brings the sums along to a larger maximum.
    __device__ __forceinline__ void raise(uint32_t power, float to, float c) {
        float d, d1, w, w1;
        exp_pair(power, m, m, reference(to), c, w, w1, d, d1);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            float s0, s1, q0, q1;
            unpack2(s[t], s0, s1);
            unpack2(add2_rn(q[t], pack2(__fmul_rn(d, s0), __fmul_rn(d, s1))), q0, q1);
            q[t] = pack2(__fmul_rn(w, q0), __fmul_rn(w, q1));
            s[t] = pack2(__fmul_rn(w, s0), __fmul_rn(w, s1));
        }
        m = to;
    }
    // A block of maximum `bm`, its first `left` columns.
    template <int TY>
    __device__ __forceinline__ void add(uint32_t power, const Raw<TY> &r, float bm, int left, float c) {
        const float to = max_nan(m, bm);
        if (m == kMinusInf) m = to;                    // nothing has been summed
        else if (!(to == m)) raise(power, to, c);
        const float ref = reference(m);
        auto step = [&](const uint32_t *w) {
#pragma unroll
            for (int t = 0; t < 8; t += 2) {
                float x0, x1, t0, t1, e0, e1;
                two_of<TY>(w, t, x0, x1);
                exp_pair(power, x0, x1, ref, c, e0, e1, t0, t1);
                s[t / 2] = add2_rn(s[t / 2], pack2(e0, e1));
                q[t / 2] = add2_rn(q[t / 2], pack2(__fmul_rn(e0, t0), __fmul_rn(e1, t1)));
            }
        };
        if (left > 768) {            // asked once: a shorter block is asked about step by step
#pragma unroll
            for (int i = 0; i < 4; ++i) step(r.w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (256 * i < left) step(r.w[i]);
        }
    }
    template <int TY>
    __device__ __forceinline__ float fold(const u64 (&v)[4]) {
        float f[8];
#pragma unroll
        for (int t = 0; t < 4; ++t) unpack2(v[t], f[2 * t], f[2 * t + 1]);
        return fold_residues<TY>(f);
    }
};

// ------------------------------------------------------------ alternatives ----

// The order of a value and its column, the lower column first among equals.  Never 0.
__device__ __forceinline__ u64 order_key(uint32_t value, uint32_t col) { return (u64(value) << 32) | (0xffffffffu - col); }
__device__ __forceinline__ float value_of(uint32_t order) {
    return __uint_as_float((order >> 31) ? order & 0x7fffffffu : ~order);
}
__device__ __forceinline__ float key_value(u64 k) { return value_of(uint32_t(k >> 32)); }
__device__ __forceinline__ uint32_t key_col(u64 k) { return 0xffffffffu - uint32_t(k); }

// The n-th largest of a warp's values: sorted by a bitonic network.
__device__ __forceinline__ uint32_t nth_largest(uint32_t v, int n) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k *= 2)
#pragma unroll
        for (int j = k / 2; j; j /= 2) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, v, j);
            v = ((lane & k) == 0) == ((lane & j) == 0) ? max(v, o) : min(v, o);
        }
    return __shfl_sync(0xffffffffu, v, n - 1);
}

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

constexpr float kLn2 = 0x1.62e430p-1f, kLn2High = 0x1.62e400p-1f, kLn2Low = 0x1.7f7d1cp-20f;

// ln of a finite S >= 1/2, of 0, or of a NaN.
__device__ __forceinline__ float ln_fixed(float S) {
    if (!(S > 0.0f)) return S == 0.0f ? kMinusInf : S;
    const uint32_t bits = __float_as_uint(S);
    int E = int(bits >> 23) - 127;
    if (E == 128) return S;
    float F = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
    if (F > 0x1.6a09e6p+0f) {
        F = __fmul_rn(F, 0.5f);
        ++E;
    }
    const float z = __fdiv_rn(__fsub_rn(F, 1.0f), __fadd_rn(F, 1.0f)), zz = __fmul_rn(z, z), r = __fadd_rn(z, z);
    float p = 1.0f / 9;
    p = __fadd_rn(__fmul_rn(p, zz), 1.0f / 7);
    p = __fadd_rn(__fmul_rn(p, zz), 1.0f / 5);
    p = __fadd_rn(__fmul_rn(p, zz), 1.0f / 3);
    const float lnF = __fadd_rn(r, __fmul_rn(r, __fmul_rn(zz, p)));
    // E * kLn2High is exact: 15 bits by 8
    return __fadd_rn(__fmul_rn(float(E), kLn2High), __fadd_rn(lnF, __fmul_rn(float(E), kLn2Low)));
}

__device__ __forceinline__ float logp_of(float x, float M, float inv, float lnS) {
    if (x == kMinusInf && M < -kMinusInf) return x;     // impossible, also where all is
    return __fsub_rn(__fmul_rn(__fsub_rn(x, M), inv), lnS);
}

// Shared memory of a row's first CTA: m, s and q of the segments, the blocks' maxima,
// and with alternatives the chosen blocks and the values to be ranked.
struct Listed {
    u64 keys[kMostListed];           // more in each warp's list where there are too many
    uint32_t chosen[kMostTop];
    uint32_t least;                  // of the chosen blocks' maxima
    int count;
    float M, lnS;
};
__host__ __device__ inline size_t lp_sums(int segments, int blocks) {
    return (size_t(segments) * 12 + size_t(blocks) * 4 + 15) / 16 * 16;
}
__host__ __device__ inline size_t lp_smem(int segments, int blocks) { return lp_sums(segments, blocks) + sizeof(Listed); }

// Position of (value, place) among n values in falling order, the lower place first.
__device__ __forceinline__ int rank_of(const uint32_t *v, int n, uint32_t value, int place) {
    int before = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) before += v[j] > value || (v[j] == value && j < place);
    return before;
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

// A cluster a row; its warps take the segments in turn, a block of 1024 columns in
// registers at a time: its maximum first, then its exponentials.  Bound by the issue of
// instructions in bfloat16 (4096 x 131072 in 322 us, 3.3 TB/s: 17 a value, of which 4.5
// work on pairs and take two slots, 92% of the issue rate), nearer to memory in binary32
// (4096 x 32768 in 92 us, 5.8 TB/s); few rows by latencies one after another (12.0 us
// for one of 131072 with 8 alternatives).
template <int TY, bool SHIFT>
__global__ void __launch_bounds__(256) logprobs_kernel(const LpArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    float *sm = reinterpret_cast<float *>(smem), *ss = sm + a.segments, *sq = ss + a.segments, *bm = sq + a.segments;
    const uint32_t *maxima = reinterpret_cast<const uint32_t *>(bm);          // by order
    Listed &l = *reinterpret_cast<Listed *>(smem + lp_sums(a.segments, a.blocks));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const uint32_t ctas = cluster_size(), rank = cluster_rank();
    if (!REPOPS_DBG_SMEM_OK(lp_smem(a.segments, a.blocks), a.status)) return;
    const int64_t row = blockIdx.x / ctas;
    constexpr int size = TY == REPOPS_TYPE_F32 ? 4 : 2;
    const int cols = int(a.cols);
    const char *x = static_cast<const char *>(a.x) + row * a.ld * size;
    const int off = SHIFT ? int(reinterpret_cast<uintptr_t>(x) % 16) / size : 0;
    uint32_t mask[4];
    if constexpr (SHIFT) slot_masks<TY>(off, mask);
    Raw<TY> v;
    const uint32_t power = kPowers[lane];
    if (ctas > 1) cluster_arrive();
    bool started = ctas == 1;
    for (int j = int(rank) * warps + warp; j < a.segments; j += int(ctas) * warps) {
        Sums sums;
        sums.clear();
        uint32_t most = 0;               // lane b's: the order of the maximum of block 4 j + b
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
            const int base = j * kSegment + b * kBlock, left = cols - base;
            if (left <= 0) break;
            load_block<TY, SHIFT>(a, x, off, mask, base, v);
            const float m = block_max<TY>(v);
            if (lane == b) most = ordered(m);
            sums.add<TY>(power, v, m, left, a.c);
        }
        const float s = sums.fold<TY>(sums.s), q = sums.fold<TY>(sums.q);
        if (!started) {              // the first CTA's shared memory is there
            cluster_wait();
            started = true;
        }
        // lanes 0 .. 3 the blocks' maxima, 4 .. 6 the segment's results
        float *to = lane < 4 ? bm + 4 * j + lane : lane == 4 ? sm + j : lane == 5 ? ss + j : sq + j;
        const float f = lane < 4 ? __uint_as_float(most) : lane == 4 ? sums.m : lane == 5 ? s : q;
        if (lane < 4 ? 4 * j + lane < a.blocks : lane < 7) {
            if (ctas > 1) store_first(to, f);
            else *to = f;
        }
    }
    if (ctas > 1) {
        if (!started) cluster_wait();
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    if (warp == 0) {
        float M = kMinusInf;
        for (int j = lane; j < a.segments; j += 32) M = max_nan(M, sm[j]);
        M = warp_max_nan(M);
        float S = 0.0f, Q = 0.0f;
        for (int j = lane; j - lane < a.segments; j += 32) {
            float t, t1, e, e1;
            const bool have = j < a.segments;
            const float m = have ? sm[j] : kMinusInf;
            exp_pair(power, m, m, reference(M), a.c, e, e1, t, t1);
            if (have) {
                S = __fadd_rn(S, __fmul_rn(e, ss[j]));
                Q = __fadd_rn(Q, __fmul_rn(e, __fadd_rn(sq[j], __fmul_rn(t, ss[j]))));
            }
        }
#pragma unroll
        for (int i = 16; i; i >>= 1) {
            S = __fadd_rn(S, __shfl_xor_sync(0xffffffffu, S, i));
            Q = __fadd_rn(Q, __shfl_xor_sync(0xffffffffu, Q, i));
        }
        if (lane == 0) {
            const bool empty = S == 0.0f;
            const int64_t t = a.targets ? load_const(a, a.targets + row) : -1;
            const float xt = t >= 0 && t < a.cols ? load_one<TY>(a, x, t) : 0.0f;
            const float lnS = ln_fixed(S);
            const float H = empty ? 0.0f : __fsub_rn(lnS, __fmul_rn(kLn2, __fdiv_rn(Q, S)));
            store_global(a, a.logp + row, t < 0 ? 0.0f : t >= a.cols ? __int_as_float(0x7fffffff) : logp_of(xt, M, a.inv, lnS));
            store_global(a, a.lse + row, empty ? M : __fadd_rn(__fmul_rn(M, a.inv), lnS));
            store_global(a, a.entropy + row, H);
            store_global(a, reinterpret_cast<float4 *>(a.stats) + row, make_float4(M, empty ? 0.0f : __frcp_rn(S), lnS, H));
            l.M = M;
            l.lnS = lnS;
        }
    }
    if (!a.top) return;
    // which blocks hold the alternatives: by counting, a thread of the warps that have no
    // sums to end for each block, or one after another by the last warp.  A step of the
    // count takes about a twelfth of finding one.  1024 rows of 32 blocks, 20 wanted, 35 us
    // and 43; 4096 such rows 109 and 119; one row of 128 blocks, 8 wanted, 12.3 either way;
    // 4096 rows of 128, 20 wanted, 350 and 345, one wanted 334 and 322
    const int chosen = min(a.top, a.blocks);
    const int others = 32;           // threads of the first warp, which has the sums
    if (warps > 1 && a.blocks < 12 * kMostTop &&
        a.blocks * ((a.blocks + others * (warps - 1) - 1) / (others * (warps - 1))) < 12 * chosen) {
        for (int b = int(threadIdx.x) - others; b >= 0 && b < a.blocks; b += int(blockDim.x) - others) {
            const uint32_t o = maxima[b];
            const int at = rank_of(maxima, a.blocks, o, b);
            if (at < chosen) l.chosen[at] = uint32_t(b);
            if (at == chosen - 1) l.least = o;
        }
    } else if (warp == warps - 1) {
        u64 before = ~u64(0);
        for (int n = 0; n < chosen; ++n) {
            u64 mine = 0;
            for (int b = lane; b < a.blocks; b += 32) {
                const u64 k = order_key(maxima[b], uint32_t(b));
                mine = (n == 0 || k < before) && k > mine ? k : mine;
            }
            const uint32_t high = __reduce_max_sync(0xffffffffu, uint32_t(mine >> 32));
            const uint32_t low = __reduce_max_sync(0xffffffffu, uint32_t(mine >> 32) == high ? uint32_t(mine) : 0u);
            before = (u64(high) << 32) | low;
            if (lane == 0) l.chosen[n] = key_col(before);
        }
        if (lane == 0) l.least = uint32_t(before >> 32);
    }
    if (threadIdx.x == 0) l.count = 0;
    __syncthreads();
    // first the values that reach the least maximum are listed and ranked; where they are
    // too many each warp keeps a list of its blocks' best (that alone: 1024 rows of 32768,
    // 20 wanted, 43.8 us instead of 33.7)
    TopList best;
#pragma unroll 1
    for (bool listed = true;; listed = false) {
        for (int n = warp; n < chosen; n += warps) {
            const int base = int(l.chosen[n]) * kBlock;
            load_block<TY, SHIFT>(a, x, off, mask, base, v);
            uint32_t least = l.least;
            if (chosen < a.top) least = nth_largest(ordered(lane_max<TY>(v)), a.top);
            const float reach = value_of(least);
            uint32_t hit = 0;            // slots whose value is not below (a NaN neither)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t = 0; t < 8; t += 2) {
                    float x0, x1;
                    two_of<TY>(v.w[i], t, x0, x1);
                    if (!(x0 < reach)) hit |= 1u << (8 * i + t);
                    if (!(x1 < reach)) hit |= 2u << (8 * i + t);
                }
            auto next = [&]() -> u64 {   // this lane's next value, or 0
                while (hit) {
                    const int e = __ffs(hit) - 1, col = base + slot_col<TY>(e >> 3, e & 7, off);
                    hit &= hit - 1;
                    if (col < cols) return order_key(ordered(load_one<TY>(a, x, col)), uint32_t(col));
                }
                return 0;
            };
            if (listed) {
                for (u64 k = next(); k; k = next()) {
                    const int at = atomicAdd(&l.count, 1);
                    if (at < kMostListed) l.keys[at] = k;
                }
            } else {
                while (__any_sync(0xffffffffu, hit != 0)) best.add(next(), a.top);
            }
        }
        __syncthreads();
        if (!listed) break;
        const int count = l.count;
        if (count > kMostListed) continue;
        for (int n = threadIdx.x; n < count; n += blockDim.x) {
            const u64 mine = l.keys[n];
            int at = 0;
            for (int j = 0; j < count; ++j) at += l.keys[j] > mine;
            if (at < a.top) {
                store_global(a, a.top_ids + row * a.top + at, int64_t(key_col(mine)));
                store_global(a, a.top_logp + row * a.top + at, logp_of(key_value(mine), l.M, a.inv, l.lnS));
            }
        }
        return;
    }
    l.keys[warp * kMostTop + lane] = best.mine;
    __syncthreads();
    if (warp == 0) {
        TopList whole;
        for (int w = 0; w < warps; ++w) whole.add(l.keys[w * kMostTop + lane], a.top);
        if (lane < a.top) {
            store_global(a, a.top_ids + row * a.top + lane, int64_t(key_col(whole.mine)));
            store_global(a, a.top_logp + row * a.top + lane, logp_of(key_value(whole.mine), l.M, a.inv, l.lnS));
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

// dx = fl(e * fl(A + fl(B * t))); at the target + G.  Four 16-byte accesses a thread
// where VEC.  Bound by memory: 4096 x 32768 binary32 read and written in 156 us (6.9
// TB/s).
template <int TY, bool ENTROPY, bool VEC>
__global__ void __launch_bounds__(256) logprobs_backward_kernel(const LpGradArgs a) {
    constexpr int N = Lanes<TY>::N, U = 4, size = 16 / N;
    const int cols = int(a.cols);
    const uint32_t power = kPowers[threadIdx.x & 31];
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const char *x = static_cast<const char *>(a.x) + row * a.ld * size;
        char *dx = static_cast<char *>(a.dx) + row * a.ldd * size;
        const int off = VEC ? int(reinterpret_cast<uintptr_t>(x) % 16) / size : 0;
        const int first = (int(blockIdx.x) * (U * 256) + int(threadIdx.x)) * N - off;
        uint32_t w[U][4];
        bool whole[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = first + u * (256 * N);
            whole[u] = VEC && col >= 0 && col + N <= cols;
            if (whole[u]) {
                const uint4 q = load_once(a, reinterpret_cast<const uint4 *>(x + int64_t(col) * size));
                w[u][0] = q.x;
                w[u][1] = q.y;
                w[u][2] = q.z;
                w[u][3] = q.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    w[u][j] = 0;
                    if constexpr (TY == REPOPS_TYPE_F32) {
                        if (col + j >= 0 && col + j < cols)
                            w[u][j] = load_global(a, reinterpret_cast<const uint32_t *>(x) + col + j);
                    } else {
                        const uint16_t *p = reinterpret_cast<const uint16_t *>(x);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (col + 2 * j + i >= 0 && col + 2 * j + i < cols)
                                w[u][j] |= uint32_t(load_global(a, p + col + 2 * j + i)) << (16 * i);
                    }
                }
            }
        }
        const float4 st = load_const(a, reinterpret_cast<const float4 *>(a.stats) + row);
        const int64_t target = a.targets ? load_const(a, a.targets + row) : -1;
        float wt = target >= 0 && a.dlogp ? load_const(a, a.dlogp + row) : 0.0f;
        if (target >= a.cols && a.dlogp) wt = __int_as_float(0x7fffffff);
        const float h = ENTROPY ? load_const(a, a.dentropy + row) : 0.0f;
        const bool empty = st.x == kMinusInf;
        const float ref = reference(st.x);
        float A = wt, B = 0.0f;
        if (ENTROPY) {
            A = __fadd_rn(A, __fmul_rn(h, __fsub_rn(st.w, st.z)));
            B = empty ? 0.0f : -__fmul_rn(__fmul_rn(__fmul_rn(a.inv, kLn2), h), st.y);
        }
        A = empty ? 0.0f : -__fmul_rn(__fmul_rn(a.inv, A), st.y);
        const float G = empty ? 0.0f : __fmul_rn(a.inv, wt);
        const int hit = target >= 0 && target < a.cols ? int(target) : -(1 << 30);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = first + u * (256 * N);
            float v[N];
#pragma unroll
            for (int t = 0; t < N; t += 2) {
                float x0, x1, e0, e1, t0, t1;
                two_of<TY>(w[u], t, x0, x1);
                exp_pair(power, x0, x1, ref, a.c, e0, e1, t0, t1);
                v[t] = __fmul_rn(e0, ENTROPY ? __fadd_rn(A, __fmul_rn(B, t0)) : A);
                v[t + 1] = __fmul_rn(e1, ENTROPY ? __fadd_rn(A, __fmul_rn(B, t1)) : A);
            }
            const int at = hit - col;
            if (at >= 0 && at < N) {
#pragma unroll
                for (int t = 0; t < N; ++t)
                    if (t == at) v[t] = __fadd_rn(v[t], G);
            }
            if (whole[u]) {
                uint4 q;
                if constexpr (TY == REPOPS_TYPE_F32) {
                    q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
                } else {
                    q = make_uint4(narrowed2<TY>(v[0], v[1]), narrowed2<TY>(v[2], v[3]), narrowed2<TY>(v[N - 4], v[N - 3]),
                                   narrowed2<TY>(v[N - 2], v[N - 1]));
                }
                store_once(a, reinterpret_cast<uint4 *>(dx + int64_t(col) * size), q);
            } else {
#pragma unroll
                for (int t = 0; t < N; ++t)
                    if (col + t >= 0 && col + t < cols) store_one<TY>(a, dx, col + t, v[t]);
            }
        }
    }
}

// ------------------------------------------------------------------- host ----

template <int TY, bool SHIFT>
int launch_logprobs(const LpArgs &a, cudaStream_t s) {
    DeviceInfo di;
    if (const int rc = current_device_info(&di); rc != REPOPS_OK) return rc;
    // Four warps a row of four segments or more: rows then end at more times than one, and
    // the others' sums fill the time (4096 rows of 131072 in bfloat16, graph-replayed: one
    // warp a row 586 us, two 346, three 335, four 322, five 332, eight 335; 4096 of 65536
    // in binary32 two 180, four 170; 20000 of 8192, two segments, one 107, two 111).  More
    // up to 32 warps an SM, a CTA's first, then, for few rows, those of a cluster's CTAs
    // (1024 rows of 131072: two 107 us, eight 94; one row by eight warps of one CTA 30 us,
    // by four CTAs 12); as few as take the same number of turns.
    int warps = a.segments >= 4 ? 4 : 1;
    unsigned ctas = 1;
    while (warps < 8 && warps < a.segments && a.rows * warps < int64_t(32) * di.sms) warps *= 2;
    while (ctas < 8 && int(ctas) * warps < a.segments && a.rows * warps * ctas < int64_t(32) * di.sms) ctas *= 2;
    if (ctas == 1) {
        const int turns = (a.segments + warps - 1) / warps;
        warps = (a.segments + turns - 1) / turns;
    }
    const size_t smem = lp_smem(a.segments, a.blocks);
    auto kern = logprobs_kernel<TY, SHIFT>;
    if (smem > 48 * 1024)
        if (const int rc = allow_shared(kern, lp_smem(int(kMostColumns / kSegment), int(kMostColumns / kBlock))); rc != REPOPS_OK)
            return rc;
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
    constexpr int tile = 4 * 256 * Lanes<TY>::N;
    const int64_t blocks = (a.cols + Lanes<TY>::N - 1 + tile - 1) / tile;
    const dim3 grid(unsigned(blocks), unsigned(std::min<int64_t>(a.rows, 65535)));
    if (a.dentropy) {
        if (vec) logprobs_backward_kernel<TY, true, true><<<grid, 256, 0, s>>>(a);
        else logprobs_backward_kernel<TY, true, false><<<grid, 256, 0, s>>>(a);
    } else {
        if (vec) logprobs_backward_kernel<TY, false, true><<<grid, 256, 0, s>>>(a);
        else logprobs_backward_kernel<TY, false, false><<<grid, 256, 0, s>>>(a);
    }
    return check_launch();
}

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
        misaligned(stats, 16) || misaligned(x, storage_size(x_type)) || misaligned(targets, 8) || misaligned(logp, 4) ||
        misaligned(lse, 4) || misaligned(entropy, 4) || (top && (misaligned(top_logp, 4) || misaligned(top_ids, 8))) ||
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
    a.inv = 1.0f / temperature;
    a.logp = logp; a.lse = lse; a.entropy = entropy; a.stats = stats;
    a.top = top; a.top_logp = top_logp; a.top_ids = top_ids;
    a.segments = int((cols + kSegment - 1) / kSegment);
    a.blocks = int((cols + kBlock - 1) / kBlock);
    a.reads(x, xb);
    a.reads(targets, uint64_t(rows) * 8u);
    for (const auto &o : outs) a.writes(o.p, o.b);
    if (const int rc = a.arm(); rc != REPOPS_OK) return rc;
    // rows that all start on 16 bytes need no shifting (in bfloat16 9 us of 356 less)
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
    if (!x || !dx || !stats || (!dlogp && !dentropy) || (dlogp && !targets) || misaligned(stats, 16) ||
        misaligned(x, size) || misaligned(dx, size) || misaligned(targets, 8) || misaligned(dlogp, 4) || misaligned(dentropy, 4) ||
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
    // every row of dx as far from a 16-byte boundary as the same row of x: 16 bytes an
    // access (156 us for 4096 x 32768, value by value 32 more)
    const bool vec = (reinterpret_cast<uintptr_t>(x) - reinterpret_cast<uintptr_t>(dx)) % 16 == 0 &&
                     (ldx - lddx) * int64_t(size) % 16 == 0;
    switch (x_type) {
        case REPOPS_TYPE_F32: return launch_backward<REPOPS_TYPE_F32>(a, vec, stream);
        case REPOPS_TYPE_F16: return launch_backward<REPOPS_TYPE_F16>(a, vec, stream);
        default: return launch_backward<REPOPS_TYPE_BF16>(a, vec, stream);
    }
}
