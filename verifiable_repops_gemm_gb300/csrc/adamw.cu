// adamw.cu -- one AdamW step over many tensors at once, from one or several
// contributors' gradients folded in a fixed order, with the moments in 32 bits
// or in 8.
//
// Per element, every step one binary32 rounding (b1' = fl(1 - beta1), b2' alike,
// c2 = fl(1 / sqrt(1 - beta2^t)), s = fl(lr / (1 - beta1^t))):
//   g     = mean of the contributors' gradients as the fixed-order mean + SGD
//           (left fold in `order`, one correctly rounded divide by their count),
//           fl(g * grad_scale) where one is given
//   m     = fl(fl(m * beta1) + fl(g * b1')),  v = fl(fl(v * beta2) + fl(fl(g * g) * b2'))
//   r     = fl(sqrt(v)),  u = fl(m / fl(fl(r * c2) + eps))
//   theta = fl(fl(theta * fl(1 - fl(decay * lr))) - fl(u * s))
// The square root is taken once: the update needs it, and the 8-bit form keeps it.
//
// 8-bit moments: m in e4m3 (sign, 4 bits of exponent, 3 of mantissa), the root r in
// 4 bits of exponent and 4 of mantissa, each with a scale 2^(s-127) for every 128
// consecutive elements of a tensor (s one byte).  The scale is the least power of
// two under which the group's largest value still has a code, so that taking it
// out and putting it back is exact and the one rounding is the code's.  beta2 moves
// v by a thousandth of itself a step, far less than half a code's width: rounded
// to the nearest code the moments would stand still.  So a value is rounded up with
// the probability that what is cut off has of passing (16 bits of a hash of the
// seed, the step, the tensor and the element: MurmurHash3's finaliser, Appleby),
// which is right on average for m and r, and the same bits on every machine.  r's
// square is not: the rounding's variance adds to v, 0.8% on the whole at beta2 = 0.95
// (normal gradients, 600 steps) and 2% at 0.999 (6000 steps), where 7% of the elements
// are 1.25 times or more too high on average over half of the run.  A root that is
// not zero keeps a code that is not zero, as m / 0 would follow; where a group's roots
// span more than 2^18 that code holds the small ones up, by orders of magnitude.  A group holding an
// infinity or a NaN gets the scale 255 and is NaN from then on.
//
// Bytes an element: 12 + 16 with moments in 32 bits, 12 + 4 + 1/32 in 8 (binary32
// gradients); no order is left open, as elements are independent and a group's
// largest value does not depend on how it is found.  32-bit moments run at the
// memory's rate (60.8 M elements 247 us, 6.9 TB/s); 8-bit ones are bound by the
// instructions of a square root, a quotient, two codes and their dither (133 an
// element with four gradients, 80% of the issue rate): 184 us with one gradient,
// 254 with four in bfloat16.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "storage.cuh"

namespace repops {
namespace {

constexpr int kGroup = 128;          // elements that share a scale
constexpr int kTile = 4096;          // elements of a CTA: 16 a thread
constexpr int kThreads = 256;

// One tensor of a launch, in 64-bit words: first tile | decay, elements (the top
// bit: every array aligned for four elements an access), theta, m, v, the two
// scales, then the gradients in the order of the fold.
constexpr int kEntryWords = 7;
constexpr uint64_t kAligned = uint64_t(1) << 63;

struct AdamHead {
    int tensors, stride;             // words of an entry: 7 + contributors
    int contributors, pow2;
    float count, inv;
    float b1, c1, b2, c2;            // beta1, fl(1 - beta1), beta2, fl(1 - beta2)
    float eps;
    float lr, step, root;            // lr, s and c2 above
    uint32_t key;
    uint32_t first_tensor;           // of this launch, in the whole call
    const uint32_t *scalars;         // device: lr, s, c2, key instead of those, or null
    const float *grad_scale;         // device, or null
    unsigned *status;                // checked build
};

// The table travels with the launch: nothing to copy, and a captured graph keeps
// it.  Two sizes, as the whole of it is copied for each launch (50 tensors: 6.8 us of the
// host's time in the small one, 8.0 in the large).
template <int WORDS>
struct AdamTable {
    AdamHead h;
    uint64_t w[WORDS];
};

struct Entry {
    int64_t n;
    bool vec;
    float decay;
    float *theta;
    void *m, *v;
    uint8_t *ms, *vs;
    const uint64_t *grads;
};

__device__ __forceinline__ uint32_t mix32(uint32_t h) {
    h = (h ^ (h >> 16)) * 0x85EBCA6Bu;
    h = (h ^ (h >> 13)) * 0xC2B2AE35u;
    return h ^ (h >> 16);
}

// A span of a tensor: what a tile may touch of one of its arrays (checked build).
struct Tile {
    int left;                        // elements of the tensor from the tile's first on
    bool vec;                        // four elements an access
    unsigned *status;
};
#define REPOPS_ADAM_OK(tile, base, size, p, bytes)                                                             \
    REPOPS_DBG_OK((DbgSpan{reinterpret_cast<uintptr_t>(base), reinterpret_cast<uintptr_t>(base) + uint64_t((tile).left) * (size)}), \
                  p, bytes, (tile).status)
// The same for a byte of the scales of n elements.
#define REPOPS_ADAM_SCALE_OK(base, n, p, status)                                                                          \
    REPOPS_DBG_OK((DbgSpan{reinterpret_cast<uintptr_t>(base), reinterpret_cast<uintptr_t>(base) + uint64_t((n) + kGroup - 1) / kGroup}), \
                  p, 1, status)

// Elements e .. e+3 of a tile, `have` of them there (0 .. 4); the others +0.  FULL: all
// four, aligned, asked about once for the tile.
template <int TY, bool FULL>
__device__ __forceinline__ float4 load4(const Tile &t, const void *base, int e, int have) {
    constexpr unsigned size = TY == REPOPS_TYPE_F32 ? 4 : 2;
    const char *p = static_cast<const char *>(base) + e * int(size);
    if (FULL || (t.vec && have == 4)) {
        if (!REPOPS_ADAM_OK(t, base, size, p, 4 * size)) return make_float4(0, 0, 0, 0);
        return load_four<TY>(DbgAccess{}, p, 0);
    }
    float v[4] = {0, 0, 0, 0};
    if constexpr (!FULL) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < have && REPOPS_ADAM_OK(t, base, size, p + i * size, size)) v[i] = load_one<TY>(DbgAccess{}, p, i);
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

template <bool FULL>
__device__ __forceinline__ void store4(const Tile &t, float *base, int e, int have, float4 v) {
    float *p = base + e;
    if (FULL || (t.vec && have == 4)) {
        if (REPOPS_ADAM_OK(t, base, 4, p, 16)) store_four<REPOPS_TYPE_F32>(DbgAccess{}, p, 0, v);
        return;
    }
    if constexpr (!FULL) {
        const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < have && REPOPS_ADAM_OK(t, base, 4, p + i, 4)) p[i] = a[i];
    }
}

template <bool FULL>
__device__ __forceinline__ uint32_t load_codes(const Tile &t, const uint8_t *base, int e, int have) {
    const uint8_t *p = base + e;
    if (FULL || (t.vec && have == 4))
        return REPOPS_ADAM_OK(t, base, 1, p, 4) ? __ldcs(reinterpret_cast<const uint32_t *>(p)) : 0u;
    uint32_t w = 0;
    if constexpr (!FULL) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < have && REPOPS_ADAM_OK(t, base, 1, p + i, 1)) w |= uint32_t(p[i]) << (8 * i);
    }
    return w;
}

template <bool FULL>
__device__ __forceinline__ void store_codes(const Tile &t, uint8_t *base, int e, int have, uint32_t w) {
    uint8_t *p = base + e;
    if (FULL || (t.vec && have == 4)) {
        if (REPOPS_ADAM_OK(t, base, 1, p, 4)) __stcs(reinterpret_cast<uint32_t *>(p), w);
        return;
    }
    if constexpr (!FULL) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < have && REPOPS_ADAM_OK(t, base, 1, p + i, 1)) p[i] = uint8_t(w >> (8 * i));
    }
}

// ------------------------------------------------------------ 8-bit codes ----

// A code's bits as the exponent and mantissa of a binary32 number are the code's
// value times a power of two, its subnormals included: exact products give it back.
// (e4m3 has conversion instructions, its values are binary16's as well.)
__device__ __forceinline__ void decode_m(uint32_t c, float scale, float4 &v) {
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(uint16_t(c)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(uint16_t(c >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    v = make_float4(__fmul_rn(a.x, scale), __fmul_rn(a.y, scale), __fmul_rn(b.x, scale), __fmul_rn(b.y, scale));
}
__device__ __forceinline__ float decode_r(uint32_t c, float scale) {
    return __fmul_rn(__fmul_rn(__uint_as_float((c & 0xffu) << 19), 0x1p+112f), scale);
}
__device__ __forceinline__ float scale_of(uint32_t s) { return __uint_as_float(s << 23); }

// s for a group whose largest magnitude has the bits `amax`: the largest code is
// 1.75 * 2^8 (m) or 1.9375 (r) times the scale.  0: the group is not finite.
template <bool ROOT>
__device__ __forceinline__ uint32_t group_scale(uint32_t amax) {
    if (amax >= 0x7f800000u) return 255u;
    const int s = int((amax + (ROOT ? 0x07ffffu : 0x1fffffu)) >> 23) - (ROOT ? 0 : 8);
    return uint32_t(max(s, 1));
}
// 2^(127 - s): normal for s up to 253 (a root's s is below 192).
__device__ __forceinline__ float inverse_scale(uint32_t s) { return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23); }

__device__ __forceinline__ uint32_t encode_m(float x, float inv, uint32_t dither) {
    const uint32_t y = __float_as_uint(__fmul_rn(__fmul_rn(fabsf(x), inv), 0x1p-120f));
    return ((y + ((dither << 4) | 8u)) >> 20) | ((__float_as_uint(x) >> 24) & 0x80u);
}
__device__ __forceinline__ uint32_t encode_r(float r, float inv, uint32_t dither) {
    const uint32_t y = __float_as_uint(__fmul_rn(__fmul_rn(r, inv), 0x1p-112f));
    const uint32_t c = (y + ((dither << 3) | 4u)) >> 19;
    return c == 0 && y != 0 ? 1u : c;
}

__device__ __forceinline__ uint32_t packed(const uint32_t (&c)[4]) {
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

// ----------------------------------------------------------------- kernel ----

struct Step {
    float b1, c1, b2, c2, eps, keep, step, root;
};

// theta, m and v (or r with 8-bit moments) of one element.
__device__ __forceinline__ void update(float &theta, float &m, float &v, float &r, float g, const Step &k) {
    m = __fadd_rn(__fmul_rn(m, k.b1), __fmul_rn(g, k.c1));
    v = __fadd_rn(__fmul_rn(v, k.b2), __fmul_rn(__fmul_rn(g, g), k.c2));
    r = __fsqrt_rn(v);
    const float u = __fdiv_rn(m, __fadd_rn(__fmul_rn(r, k.root), k.eps));
    theta = __fsub_rn(__fmul_rn(theta, k.keep), __fmul_rn(u, k.step));
}

__device__ __forceinline__ void add4(float4 &a, float4 b) {
    a.x = __fadd_rn(a.x, b.x);
    a.y = __fadd_rn(a.y, b.y);
    a.z = __fadd_rn(a.z, b.z);
    a.w = __fadd_rn(a.w, b.w);
}

// CTAs an SM: 8-bit moments and several gradients hide their loads behind many warps of
// one vector a thread (60.8 M elements, four binary32 gradients: 343 us with 32-bit
// moments, 250 with 8-bit; two vectors and four CTAs: 359 and 274); one gradient and
// 32-bit moments behind two vectors (245 us either way).
template <bool EIGHT, bool MANY>
constexpr int kCtas = EIGHT || MANY ? 5 : 1;

// U vectors of four elements a thread are in flight together, and with several
// contributors those of four of them.  FULL: a whole tile of aligned tensors (60.8 M
// elements with 32-bit moments 247 us, asked about vector by vector 250, value by value
// 254; 8-bit moments and four gradients in bfloat16, with the moments restored: 353, 457
// and 606).
template <int TY, bool EIGHT, bool MANY, bool FULL>
__device__ __forceinline__ void run_tile(const AdamHead &h, const Entry &t, int64_t base, const Step &k, uint32_t key,
                                         float gscale, bool scaled) {
    constexpr int U = EIGHT || MANY ? 1 : 2, kPart = kThreads * 4 * U;
    constexpr unsigned gsize = TY == REPOPS_TYPE_F32 ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const Tile tile{int(min(int64_t(kTile), t.n - base)), t.vec, h.status};
    float *theta_at = t.theta + base;
    char *m_at = static_cast<char *>(t.m) + base * (EIGHT ? 1 : 4), *v_at = static_cast<char *>(t.v) + base * (EIGHT ? 1 : 4);
    uint8_t *ms_at = t.ms + base / kGroup, *vs_at = t.vs + base / kGroup;
    // a tile's scales, read and written at once: a byte here and there of lines that other
    // CTAs write to as well cost microseconds each
    constexpr int kScales = kTile / kGroup;
    __shared__ uint32_t scales[2][kScales];
    const int groups = (tile.left + kGroup - 1) / kGroup;
    if constexpr (EIGHT) {
        if (int(threadIdx.x) < 2 * kScales) {
            const int i = threadIdx.x % kScales;
            const uint8_t *p = (int(threadIdx.x) < kScales ? ms_at : vs_at) + i;
            scales[threadIdx.x / kScales][i] =
                i < groups && REPOPS_ADAM_SCALE_OK(int(threadIdx.x) < kScales ? t.ms : t.vs, t.n, p, h.status) ? *p : 0;
        }
        __syncthreads();
    }
    const int64_t gradient_at = base * gsize;
    auto gradient = [&](int c) { return reinterpret_cast<const char *>(t.grads[c]) + gradient_at; };
#pragma unroll 1
    for (int part = 0; part < kTile; part += kPart) {
        if (!FULL && part >= tile.left) break;                   // the same for the whole CTA
        const int first = part + int(threadIdx.x) * 4;
        float4 theta[U], g[U], m[U], v[U];
        uint32_t mc[U], vc[U], ms[U], vs[U];
        int have[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int e = first + j * (kThreads * 4);
            have[j] = FULL ? 4 : max(0, min(4, tile.left - e));
            g[j] = load4<TY, FULL>(tile, gradient(0), e, have[j]);
            theta[j] = load4<REPOPS_TYPE_F32, FULL>(tile, theta_at, e, have[j]);
            if constexpr (EIGHT) {
                mc[j] = load_codes<FULL>(tile, reinterpret_cast<uint8_t *>(m_at), e, have[j]);
                vc[j] = load_codes<FULL>(tile, reinterpret_cast<uint8_t *>(v_at), e, have[j]);
                ms[j] = scales[0][e / kGroup];
                vs[j] = scales[1][e / kGroup];
            } else {
                m[j] = load4<REPOPS_TYPE_F32, FULL>(tile, m_at, e, have[j]);
                v[j] = load4<REPOPS_TYPE_F32, FULL>(tile, v_at, e, have[j]);
            }
        }
        if constexpr (MANY) {
            constexpr int B = 4;
            for (int c = 1; c < h.contributors; c += B) {
                float4 w[B][U];
#pragma unroll
                for (int i = 0; i < B; ++i)
                    if (c + i < h.contributors)
#pragma unroll
                        for (int j = 0; j < U; ++j)
                            w[i][j] = load4<TY, FULL>(tile, gradient(c + i), first + j * (kThreads * 4), have[j]);
#pragma unroll
                for (int i = 0; i < B; ++i)
                    if (c + i < h.contributors)
#pragma unroll
                        for (int j = 0; j < U; ++j) add4(g[j], w[i][j]);
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int e = first + j * (kThreads * 4);
            float *gj = &g[j].x, *tj = &theta[j].x, *mj = &m[j].x, *vj = &v[j].x;
            float r[4];
            if constexpr (EIGHT) {
                decode_m(mc[j], scale_of(ms[j]), m[j]);
                const float rs = scale_of(vs[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float was = decode_r(vc[j] >> (8 * i), rs);
                    vj[i] = __fmul_rn(was, was);
                }
            }
            if (MANY && !h.pow2) {
#pragma unroll
                for (int i = 0; i < 4; ++i) gj[i] = __fdiv_rn(gj[i], h.count);
            } else if (MANY) {
#pragma unroll
                for (int i = 0; i < 4; ++i) gj[i] = __fmul_rn(gj[i], h.inv);
            }
            if (scaled) {
#pragma unroll
                for (int i = 0; i < 4; ++i) gj[i] = __fmul_rn(gj[i], gscale);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) update(tj[i], mj[i], vj[i], r[i], gj[i], k);
            if (FULL || have[j]) store4<FULL>(tile, theta_at, e, have[j], theta[j]);
            if constexpr (EIGHT) {
                uint32_t am = 0, ar = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    am = max(am, FULL || i < have[j] ? __float_as_uint(mj[i]) & 0x7fffffffu : 0u);
                    ar = max(ar, FULL || i < have[j] ? __float_as_uint(r[i]) & 0x7fffffffu : 0u);
                }
                const uint32_t sm = group_scale<false>(__reduce_max_sync(0xffffffffu, am));
                const uint32_t sr = group_scale<true>(__reduce_max_sync(0xffffffffu, ar));
                const float im = inverse_scale(sm), ir = inverse_scale(sr);
                uint32_t cm[4], cr[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t d = mix32(uint32_t(base + e + i) * 0x9E3779B1u + key);
                    cm[i] = encode_m(mj[i], im, d & 0xffffu);
                    cr[i] = encode_r(r[i], ir, d >> 16);
                }
                if (FULL || have[j]) {
                    store_codes<FULL>(tile, reinterpret_cast<uint8_t *>(m_at), e, have[j], sm == 255u ? 0u : packed(cm));
                    store_codes<FULL>(tile, reinterpret_cast<uint8_t *>(v_at), e, have[j], sr == 255u ? 0u : packed(cr));
                    if (lane == 0) {         // read by this warp alone, which has its own groups
                        scales[0][e / kGroup] = sm;
                        scales[1][e / kGroup] = sr;
                    }
                }
            } else if (FULL || have[j]) {
                store4<FULL>(tile, reinterpret_cast<float *>(m_at), e, have[j], m[j]);
                store4<FULL>(tile, reinterpret_cast<float *>(v_at), e, have[j], v[j]);
            }
        }
    }
    if constexpr (EIGHT) {
        __syncthreads();
        if (int(threadIdx.x) < 2 * kScales) {
            const int i = threadIdx.x % kScales;
            uint8_t *p = (int(threadIdx.x) < kScales ? ms_at : vs_at) + i;
            if (i < groups && REPOPS_ADAM_SCALE_OK(int(threadIdx.x) < kScales ? t.ms : t.vs, t.n, p, h.status))
                *p = uint8_t(scales[threadIdx.x / kScales][i]);
        }
    }
}

template <int TY, bool EIGHT, bool MANY, int WORDS>
__global__ void __launch_bounds__(kThreads, kCtas<EIGHT, MANY>) adamw_kernel(const __grid_constant__ AdamTable<WORDS> a) {
    const AdamHead &h = a.h;
    // the tensor whose tiles hold this one
    int lo = 0, hi = h.tensors - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (uint32_t(a.w[mid * h.stride]) <= blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const uint64_t *w = a.w + lo * h.stride;
    Entry t;
    t.n = int64_t(w[1] & ~kAligned);
    t.vec = (w[1] & kAligned) != 0;
    t.decay = __uint_as_float(uint32_t(w[0] >> 32));
    t.theta = reinterpret_cast<float *>(w[2]);
    t.m = reinterpret_cast<void *>(w[3]);
    t.v = reinterpret_cast<void *>(w[4]);
    t.ms = reinterpret_cast<uint8_t *>(w[5]);
    t.vs = reinterpret_cast<uint8_t *>(w[6]);
    t.grads = w + kEntryWords;
    float lr = h.lr, step = h.step, root = h.root;
    uint32_t key = h.key;
    if (h.scalars) {
        lr = __uint_as_float(__ldg(h.scalars));
        step = __uint_as_float(__ldg(h.scalars + 1));
        root = __uint_as_float(__ldg(h.scalars + 2));
        key = __ldg(h.scalars + 3);
    }
    const Step k{h.b1, h.c1, h.b2, h.c2, h.eps, __fsub_rn(1.0f, __fmul_rn(t.decay, lr)), step, root};
    key = mix32(key + 0x9E3779B9u * (h.first_tensor + uint32_t(lo) + 1u));
    const float gscale = h.grad_scale ? __ldg(h.grad_scale) : 1.0f;
    const int64_t base = int64_t(blockIdx.x - uint32_t(w[0])) * kTile;
    if (t.vec && base + kTile <= t.n) run_tile<TY, EIGHT, MANY, true>(h, t, base, k, key, gscale, h.grad_scale != nullptr);
    else run_tile<TY, EIGHT, MANY, false>(h, t, base, k, key, gscale, h.grad_scale != nullptr);
}

// m and v of 8-bit moments as the binary32 values they stand for.
__global__ void __launch_bounds__(kThreads)
adamw_moments_kernel(int64_t n, const uint8_t *m, const uint8_t *v, const uint8_t *ms, const uint8_t *vs, float *m_out,
                     float *v_out, int vec, unsigned *status) {
    const int64_t step = int64_t(gridDim.x) * kThreads * 4;
    for (int64_t e = (blockIdx.x * int64_t(kThreads) + threadIdx.x) * 4; e < n; e += step) {
        const int have = int(min(int64_t(4), n - e));
        const Tile t{int(min(n - e, int64_t(1) << 20)), vec != 0, status};
        const uint32_t mc = load_codes<false>(t, m + e, 0, have), vc = load_codes<false>(t, v + e, 0, have);
        float4 x, y;
        const bool in = REPOPS_ADAM_SCALE_OK(ms, n, ms + e / kGroup, status) && REPOPS_ADAM_SCALE_OK(vs, n, vs + e / kGroup, status);
        decode_m(mc, in ? scale_of(__ldg(ms + e / kGroup)) : 0.0f, x);
        const float rs = in ? scale_of(__ldg(vs + e / kGroup)) : 0.0f;
        float *py = &y.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float r = decode_r(vc >> (8 * i), rs);
            py[i] = __fmul_rn(r, r);
        }
        store4<false>(t, m_out + e, 0, have, x);
        store4<false>(t, v_out + e, 0, have, y);
    }
}

// ------------------------------------------------------------------- host ----

constexpr int kSmallWords = 448, kLargeWords = 3968;     // 3.6 and 31.1 KB of kernel parameters

template <int TY, bool EIGHT, bool MANY>
int launch(const AdamHead &h, const std::vector<uint64_t> &w, unsigned tiles, cudaStream_t s) {
    if (w.size() <= size_t(kSmallWords)) {
        AdamTable<kSmallWords> a;
        a.h = h;
        std::copy(w.begin(), w.end(), a.w);
        adamw_kernel<TY, EIGHT, MANY, kSmallWords><<<tiles, kThreads, 0, s>>>(a);
    } else {
        AdamTable<kLargeWords> a;
        a.h = h;
        std::copy(w.begin(), w.end(), a.w);
        adamw_kernel<TY, EIGHT, MANY, kLargeWords><<<tiles, kThreads, 0, s>>>(a);
    }
    return check_launch();
}

template <int TY>
int launch_typed(const AdamHead &h, const std::vector<uint64_t> &w, unsigned tiles, bool eight, cudaStream_t s) {
    if (eight) return h.contributors > 1 ? launch<TY, true, true>(h, w, tiles, s) : launch<TY, true, false>(h, w, tiles, s);
    return h.contributors > 1 ? launch<TY, false, true>(h, w, tiles, s) : launch<TY, false, false>(h, w, tiles, s);
}

struct Range {
    uintptr_t lo, hi;
    bool written;
    bool operator<(const Range &o) const { return lo < o.lo; }
};

// Whether a written range shares a byte with any other.
bool ranges_clash(std::vector<Range> &r) {
    // lists of tensors mostly come in a few ascending stretches, which merge quicker than
    // they sort
    std::vector<size_t> cut{0}, next;
    for (size_t i = 1; i < r.size(); ++i)
        if (r[i] < r[i - 1]) cut.push_back(i);
    cut.push_back(r.size());
    while (cut.size() > 2) {
        next.assign(1, 0);
        for (size_t k = 0; k + 1 < cut.size(); k += 2) {
            const size_t last = std::min(k + 2, cut.size() - 1);
            if (last == k + 2)
                std::inplace_merge(r.begin() + ptrdiff_t(cut[k]), r.begin() + ptrdiff_t(cut[k + 1]), r.begin() + ptrdiff_t(cut[last]));
            next.push_back(cut[last]);
        }
        cut.swap(next);
    }
    uintptr_t end = 0, written_end = 0;
    for (const Range &x : r) {
        if (x.lo < written_end || (x.written && x.lo < end)) return true;
        end = std::max(end, x.hi);
        if (x.written) written_end = std::max(written_end, x.hi);
    }
    return false;
}

// b^n by squaring: IEEE products alone, the same bits on any host.
double power(double b, uint64_t n) {
    double p = 1.0;
    for (; n; n >>= 1, b *= b)
        if (n & 1) p *= b;
    return p;
}

uint32_t mix32_host(uint32_t h) {
    h = (h ^ (h >> 16)) * 0x85EBCA6Bu;
    h = (h ^ (h >> 13)) * 0xC2B2AE35u;
    return h ^ (h >> 16);
}

bool in_unit(double b) { return b >= 0.0 && b < 1.0; }

}  // namespace
}  // namespace repops

using namespace repops;

extern "C" int repops_adamw_scalars(int64_t step, const double *rates, uint32_t seed, uint32_t *scalars) {
    if (!rates) return REPOPS_ERR_INVALID_ARG;
    const double lr = rates[0], beta1 = rates[1], beta2 = rates[2];
    if (step < 1 || !in_unit(beta1) || !in_unit(beta2) || !std::isfinite(lr) || !scalars) return REPOPS_ERR_INVALID_ARG;
    const float f[3] = {float(lr), float(lr / (1.0 - power(beta1, uint64_t(step)))),
                        float(1.0 / std::sqrt(1.0 - power(beta2, uint64_t(step))))};
    std::memcpy(scalars, f, sizeof f);
    scalars[3] = mix32_host(0x9E3779B9u * uint32_t(step) + seed);
    return REPOPS_OK;
}

extern "C" int repops_adamw(int tensors, const int64_t *sizes, float *const *theta, int contributors,
                            const void *const *grads, int grad_type, const int *order, void *const *m, void *const *v,
                            uint8_t *const *m_scale, uint8_t *const *v_scale, const float *decay,
                            const double *hyper, const uint32_t *scalars, int scalars_on_device,
                            const float *grad_scale, cudaStream_t stream) try {
    if (!hyper) return REPOPS_ERR_INVALID_ARG;
    const double beta1 = hyper[0], beta2 = hyper[1], eps = hyper[2];
    if (tensors < 0 || contributors < 1 || contributors > REPOPS_MEAN_MAX_CONTRIBUTORS || !known_storage(grad_type) ||
        !in_unit(beta1) || !in_unit(beta2) || !(eps >= 0.0) || !scalars || !order ||
        (m_scale != nullptr) != (v_scale != nullptr))
        return REPOPS_ERR_INVALID_ARG;
    std::vector<char> seen(size_t(contributors), 0);
    for (int c = 0; c < contributors; ++c) {
        if (order[c] < 0 || order[c] >= contributors || seen[size_t(order[c])]) return REPOPS_ERR_ORDER;
        seen[size_t(order[c])] = 1;
    }
    if (tensors == 0) return REPOPS_OK;
    if (!sizes || !theta || !grads || !m || !v) return REPOPS_ERR_INVALID_ARG;
    const bool eight = m_scale != nullptr;
    const unsigned gsize = storage_size(grad_type), ssize = eight ? 1u : 4u;
    for (int i = 0; i < tensors; ++i) {
        const int64_t n = sizes[i];
        if (n < 0 || n > (int64_t(1) << 40)) return REPOPS_ERR_INVALID_ARG;
        if (n == 0) continue;
        if (!theta[i] || !m[i] || !v[i] || (eight && (!m_scale[i] || !v_scale[i]))) return REPOPS_ERR_INVALID_ARG;
        if (misaligned(theta[i], 4) || misaligned(m[i], ssize) || misaligned(v[i], ssize)) return REPOPS_ERR_INVALID_ARG;
        for (int c = 0; c < contributors; ++c) {
            const void *g = grads[int64_t(i) * contributors + c];
            if (!g || misaligned(g, gsize)) return REPOPS_ERR_INVALID_ARG;
        }
    }
    if (misaligned(scalars, 4) || misaligned(grad_scale, 4)) return REPOPS_ERR_INVALID_ARG;
    std::vector<Range> ranges;
    ranges.reserve(size_t(tensors) * size_t(5 + contributors) + 2);
    auto range = [&](const void *p, uint64_t bytes, bool written) {
        ranges.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, written});
    };
    auto list = [&](auto p, int stride, bool written, auto bytes) {
        for (int i = 0; i < tensors; ++i)
            if (sizes[i]) range(p[int64_t(i) * stride], bytes(uint64_t(sizes[i])), written);
    };
    auto group_bytes = [](uint64_t n) { return (n + kGroup - 1) / kGroup; };
    list(theta, 1, true, [](uint64_t n) { return n * 4u; });
    list(m, 1, true, [&](uint64_t n) { return n * ssize; });
    list(v, 1, true, [&](uint64_t n) { return n * ssize; });
    if (eight) {
        list(m_scale, 1, true, group_bytes);
        list(v_scale, 1, true, group_bytes);
    }
    for (int c = 0; c < contributors; ++c) list(grads + c, contributors, false, [&](uint64_t n) { return n * gsize; });
    if (ranges.empty()) return REPOPS_OK;
    if (scalars_on_device) range(scalars, 16, false);
    if (grad_scale) range(grad_scale, 4, false);
    if (ranges_clash(ranges)) return REPOPS_ERR_ALIAS;

    AdamHead h{};
    h.stride = kEntryWords + contributors;
    h.contributors = contributors;
    h.pow2 = (contributors & (contributors - 1)) == 0;
    h.count = float(contributors);
    h.inv = h.pow2 ? 1.0f / float(contributors) : 0.0f;
    h.b1 = float(beta1);
    h.c1 = float(1.0 - beta1);
    h.b2 = float(beta2);
    h.c2 = float(1.0 - beta2);
    h.eps = float(eps);
    if (scalars_on_device) {
        h.scalars = scalars;
    } else {
        float f[3];
        std::memcpy(f, scalars, sizeof f);
        h.lr = f[0];
        h.step = f[1];
        h.root = f[2];
        h.key = scalars[3];
    }
    h.grad_scale = grad_scale;
    if (const int rc = status_word_address(&h.status); rc != REPOPS_OK) return rc;

    std::vector<uint64_t> w;
    w.reserve(size_t(std::min(int64_t(tensors) * h.stride, int64_t(kLargeWords))));
    int64_t tiles = 0;
    int rc = REPOPS_OK;
    auto flush = [&](int next) {
        if (tiles && rc == REPOPS_OK) {      // a table may hold empty tensors alone
            switch (grad_type) {
                case REPOPS_TYPE_F32: rc = launch_typed<REPOPS_TYPE_F32>(h, w, unsigned(tiles), eight, stream); break;
                case REPOPS_TYPE_F16: rc = launch_typed<REPOPS_TYPE_F16>(h, w, unsigned(tiles), eight, stream); break;
                default: rc = launch_typed<REPOPS_TYPE_BF16>(h, w, unsigned(tiles), eight, stream); break;
            }
        }
        h.tensors = 0;
        h.first_tensor = uint32_t(next);
        w.clear();
        tiles = 0;
    };
    for (int i = 0; i < tensors && rc == REPOPS_OK; ++i) {
        const int64_t n = sizes[i], more = (n + kTile - 1) / kTile;
        // a launch's tensors are consecutive ones of the call; an empty one keeps its place
        if (w.size() + size_t(h.stride) > size_t(kLargeWords) || tiles + more > INT32_MAX) flush(i);
        uintptr_t bits = reinterpret_cast<uintptr_t>(theta[i]);
        bits |= (reinterpret_cast<uintptr_t>(m[i]) | reinterpret_cast<uintptr_t>(v[i])) * (eight ? 4u : 1u);
        for (int c = 0; c < contributors; ++c)
            bits |= reinterpret_cast<uintptr_t>(grads[int64_t(i) * contributors + c]) * (4u / gsize);
        uint32_t d = 0;
        if (decay) std::memcpy(&d, decay + i, 4);
        w.push_back(uint64_t(uint32_t(tiles)) | (uint64_t(d) << 32));
        w.push_back(uint64_t(n) | (bits % 16 == 0 ? kAligned : 0));
        w.push_back(reinterpret_cast<uint64_t>(theta[i]));
        w.push_back(reinterpret_cast<uint64_t>(m[i]));
        w.push_back(reinterpret_cast<uint64_t>(v[i]));
        w.push_back(eight ? reinterpret_cast<uint64_t>(m_scale[i]) : 0);
        w.push_back(eight ? reinterpret_cast<uint64_t>(v_scale[i]) : 0);
        for (int c = 0; c < contributors; ++c)
            w.push_back(reinterpret_cast<uint64_t>(grads[int64_t(i) * contributors + order[c]]));
        ++h.tensors;
        tiles += more;
    }
    if (tiles) flush(tensors);
    return rc;
} catch (const std::bad_alloc &) {       // before the first launch: the table is reserved in full
    return REPOPS_ERR_ALLOC;
}

extern "C" int repops_adamw_moments(int64_t n, const uint8_t *m, const uint8_t *v, const uint8_t *m_scale,
                                    const uint8_t *v_scale, float *m_out, float *v_out, cudaStream_t stream) {
    if (n < 0 || n > (int64_t(1) << 40)) return REPOPS_ERR_INVALID_ARG;
    if (n == 0) return REPOPS_OK;
    if (!m || !v || !m_scale || !v_scale || !m_out || !v_out || misaligned(m_out, 4) || misaligned(v_out, 4))
        return REPOPS_ERR_INVALID_ARG;
    const uint64_t groups = uint64_t(n + kGroup - 1) / kGroup, bytes = uint64_t(n) * 4u;
    for (const auto &in : {std::pair<const void *, uint64_t>{m, uint64_t(n)}, {v, uint64_t(n)}, {m_scale, groups}, {v_scale, groups}})
        if (ranges_overlap(m_out, bytes, in.first, in.second) || ranges_overlap(v_out, bytes, in.first, in.second))
            return REPOPS_ERR_ALIAS;
    if (ranges_overlap(m_out, bytes, v_out, bytes)) return REPOPS_ERR_ALIAS;
    unsigned *status;
    if (const int rc = status_word_address(&status); rc != REPOPS_OK) return rc;
    DeviceInfo di;
    if (const int rc = current_device_info(&di); rc != REPOPS_OK) return rc;
    const uintptr_t bits = ((reinterpret_cast<uintptr_t>(m) | reinterpret_cast<uintptr_t>(v)) * 4u) |
                           reinterpret_cast<uintptr_t>(m_out) | reinterpret_cast<uintptr_t>(v_out);
    const int64_t units = (n + 4 * kThreads - 1) / (4 * kThreads);
    adamw_moments_kernel<<<unsigned(std::min<int64_t>(units, int64_t(di.sms) * 32)), kThreads, 0, stream>>>(
        n, m, v, m_scale, v_scale, m_out, v_out, bits % 16 == 0, status);
    return check_launch();
}
