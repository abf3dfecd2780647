// rows8.cu -- activations kept in 8 bits: rows quantised with a scale for each
// group of columns, restored, and SwiGLU's backward read straight from them.
//
// Format, for every group of a row, each step one binary32 rounding:
//   amax = max |x|,  a = max(amax, 2^-100),
//   scale = min(fl(a / 127), S),  q = rint(fl(x * fl(127 / a))) (ties to even);
// |x| <= a, so fl(x * fl(127 / a)) <= 127 * (1 + 2^-23) and rint gives at most
// 127: no clamp.  The floor keeps 127 / a finite: a group below it is kept in
// whole parts of the floor's scale, an error of at most half of one.  S is the
// largest scale that 127 times is finite, and only the largest binary32 value
// meets it: fl(a / 127) rounds up there, and it would come back as an infinity.
// S is one unit of the last place less, which moves 127 of it by 2^-16 of a scale.
// A group holding an infinity or a NaN gets scale NaN and q = 0, so it comes back
// as NaN instead of as wrong numbers.
// The maximum does not depend on the order it is taken in, so neither does any
// bit here.
//
// All kernels stream: they are bound by memory.  Bytes an element: quantising
// 4 (or 2) + 1, restoring 1 + 4, the backward 2 + 4 in and 12 out.  4096 x 16384
// binary32 in groups of 128: 48 us to quantise and 49 to restore, 6.9 TB/s; the
// backward of 4096 x 8192 92 us, 6.6 TB/s.  Rows that do not start on 16 bytes
// move a value an instruction: 4096 x 2047 saved and restored 33 us, where
// 4096 x 2048 takes 15.
#include <algorithm>

#include "internal.cuh"
#include "rows8.cuh"
#include "swiglu.cuh"

namespace repops {
namespace {

constexpr float kScaleFloor = 0x1p-100f;
constexpr float kScaleMost = 0x1.020406p+121f;

template <int TY>
__device__ __forceinline__ float load_one(const DbgAccess &d, const void *p, int64_t i) {
    if constexpr (TY == REPOPS_TYPE_F32) return load_global(d, static_cast<const float *>(p) + i);
    else if constexpr (TY == REPOPS_TYPE_F16) return __half2float(load_global(d, static_cast<const __half *>(p) + i));
    else return __bfloat162float(load_global(d, static_cast<const __nv_bfloat16 *>(p) + i));
}

// A value as it is stored: 32 bits, or 16 in the low half.
template <int TY>
__device__ __forceinline__ uint32_t narrowed(float v) {
    if constexpr (TY == REPOPS_TYPE_F32) return __float_as_uint(v);
    else if constexpr (TY == REPOPS_TYPE_F16) return __half_as_ushort(__float2half_rn(v));
    else return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <int TY>
__device__ __forceinline__ void store_one(const DbgAccess &d, void *p, int64_t i, float v) {
    if constexpr (TY == REPOPS_TYPE_F32) store_global(d, static_cast<float *>(p) + i, v);
    else store_global(d, static_cast<uint16_t *>(p) + i, uint16_t(narrowed<TY>(v)));
}

// Elements i .. i+3, i a multiple of 4 elements from an aligned base.
template <int TY>
__device__ __forceinline__ float4 load_four(const DbgAccess &d, const void *p, int64_t i) {
    if constexpr (TY == REPOPS_TYPE_F32) {
        return load_once(d, reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
    } else {
        const uint2 w = load_once(d, reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i));
        if constexpr (TY == REPOPS_TYPE_BF16) {
            return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                               __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
        } else {
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
            return make_float4(a.x, a.y, b.x, b.y);
        }
    }
}

template <int TY>
__device__ __forceinline__ void store_four(const DbgAccess &d, void *p, int64_t i, float4 v) {
    if constexpr (TY == REPOPS_TYPE_F32) {
        store_once(d, reinterpret_cast<float4 *>(static_cast<float *>(p) + i), v);
    } else {
        store_once(d, reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i),
                   make_uint2(narrowed<TY>(v.x) | (narrowed<TY>(v.y) << 16), narrowed<TY>(v.z) | (narrowed<TY>(v.w) << 16)));
    }
}

// The larger magnitude, a NaN winning over everything.
__device__ __forceinline__ float max_mag(float m, float v) {
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(fabsf(v)));
    return m;
}
__device__ __forceinline__ float max_mag4(float m, float4 v) {
    return max_mag(max_mag(max_mag(max_mag(m, v.x), v.y), v.z), v.w);
}

struct GroupScale {
    float scale, inv;
    uint32_t keep;      // all bits, or none for a group with an infinity or a NaN
};

__device__ __forceinline__ GroupScale group_scale(float amax) {
    if (!(amax <= 3.402823466e38f)) return {__uint_as_float(0x7fffffffu), 0.0f, 0u};
    const float a = fmaxf(amax, kScaleFloor);
    return {fminf(__fdiv_rn(a, 127.0f), kScaleMost), __fdiv_rn(127.0f, a), 0xffffffffu};
}

// rint(fl(x * inv)) in the low byte: adding 1.5 * 2^23 rounds to a whole number
// (ties to even) and leaves it, two's complement, in the low mantissa bits.
__device__ __forceinline__ uint32_t quant1(float x, float inv) {
    return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.0f));
}

__device__ __forceinline__ uint32_t quant4(float4 v, const GroupScale &g) {
    const uint32_t lo = __byte_perm(quant1(v.x, g.inv), quant1(v.y, g.inv), 0x0040);
    const uint32_t hi = __byte_perm(quant1(v.z, g.inv), quant1(v.w, g.inv), 0x0040);
    return __byte_perm(lo, hi, 0x5410) & g.keep;
}

// Groups of 32 .. 256 columns: 16 values a lane, so a group is 2 to 16 lanes
// and its maximum 1 to 4 shuffles; a warp takes 512 columns of a row.  Value i
// = 4j + t of lane l of a group is its column 4 * (l + lanes * j) + t with
// 16-byte rows (VEC), else l + lanes * i, so that neighbouring lanes hold
// neighbouring columns.  Loads take no branch: a column past the row reads its
// group's first (or the row's, for a group past it), which changes no maximum.
template <int TY, bool VEC>
__global__ void __launch_bounds__(256)
quantize_groups_kernel(int64_t rows, int cols, const void *__restrict__ x, int64_t ldx, int group,
                       int8_t *__restrict__ q, int64_t ldq, float *__restrict__ scale, int64_t lds, DbgAccess dbg) {
    const int lane = threadIdx.x & 31, lanes = group / 16, l = lane & (lanes - 1);
    const int segs = (cols + 511) / 512;
    const int64_t items = rows * segs, stride = int64_t(gridDim.x) * 8;
    for (int64_t it = blockIdx.x * int64_t(8) + (threadIdx.x >> 5); it < items; it += stride) {
        const int64_t r = items <= UINT32_MAX ? uint32_t(it) / uint32_t(segs) : it / segs;
        const int g0 = int(it - r * segs) * 512 + (lane - l) * 16;      // the group's first column
        const int safe = g0 < cols ? g0 : 0;
        const int64_t base = r * ldx;
        float4 v[4];
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (VEC) {
                const int c = g0 + 4 * (l + lanes * j);
                v[j] = load_four<TY>(dbg, x, base + (c < cols ? c : safe));
            } else {
                const int c = g0 + l + 4 * lanes * j;
                v[j].x = load_one<TY>(dbg, x, base + (c < cols ? c : safe));
                v[j].y = load_one<TY>(dbg, x, base + (c + lanes < cols ? c + lanes : safe));
                v[j].z = load_one<TY>(dbg, x, base + (c + 2 * lanes < cols ? c + 2 * lanes : safe));
                v[j].w = load_one<TY>(dbg, x, base + (c + 3 * lanes < cols ? c + 3 * lanes : safe));
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max_mag4(m, v[j]);
        for (int o = lanes / 2; o > 0; o >>= 1) m = max_mag(m, __shfl_xor_sync(0xffffffffu, m, o));
        const GroupScale gs = group_scale(m);
        int8_t *o = q + r * ldq;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = quant4(v[j], gs);
            if constexpr (VEC) {
                const int c = g0 + 4 * (l + lanes * j);
                if (c < cols) store_global(dbg, reinterpret_cast<uint32_t *>(o + c), w);
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int c = g0 + l + lanes * (4 * j + t);
                    if (c < cols) store_global(dbg, o + c, int8_t(w >> (8 * t)));
                }
            }
        }
        if (l == 0 && g0 < cols) store_global(dbg, scale + r * lds + g0 / group, gs.scale);
    }
}

// One scale a row: T threads a row, each keeping up to 32 of the row's values in
// registers between the maximum and the quantisation; rows of more than 8192
// values are read again from the cache.
template <int TY, bool VEC, int T>
__global__ void __launch_bounds__(256)
quantize_rows_kernel(int64_t rows, int cols, const void *__restrict__ x, int64_t ldx, int8_t *__restrict__ q,
                     int64_t ldq, float *__restrict__ scale, int64_t lds, DbgAccess dbg) {
    constexpr int KEEP = 8, ROWS = 256 / T;
    __shared__ float part[8];
    const int t = threadIdx.x % T;
    const int steps = (cols + 4 * T - 1) / (4 * T);
    for (int64_t r0 = blockIdx.x * int64_t(ROWS); r0 < rows; r0 += int64_t(gridDim.x) * ROWS) {
        const bool live = r0 + threadIdx.x / T < rows;
        const int64_t r = live ? r0 + threadIdx.x / T : rows - 1, base = r * ldx;
        // step k covers columns [4T * k, 4T * (k + 1)): four in a row a thread
        // with 16-byte rows, else four T apart; past the end column 0 is read
        auto load = [&](int k) {
            if constexpr (VEC) {
                const int c = 4 * T * k + 4 * t;
                return load_four<TY>(dbg, x, base + (c < cols ? c : 0));
            } else {
                const int c = 4 * T * k + t;
                return make_float4(load_one<TY>(dbg, x, base + (c < cols ? c : 0)),
                                   load_one<TY>(dbg, x, base + (c + T < cols ? c + T : 0)),
                                   load_one<TY>(dbg, x, base + (c + 2 * T < cols ? c + 2 * T : 0)),
                                   load_one<TY>(dbg, x, base + (c + 3 * T < cols ? c + 3 * T : 0)));
            }
        };
        float4 v[KEEP];
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (k < steps) v[k] = load(k);
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (k < steps) m = max_mag4(m, v[k]);
        for (int k = KEEP; k < steps; ++k) m = max_mag4(m, load(k));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = max_mag(m, __shfl_xor_sync(0xffffffffu, m, o));
        if constexpr (T > 32) {
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < T / 32; ++w) m = max_mag(m, part[threadIdx.x / T * (T / 32) + w]);
            __syncthreads();
        }
        if (!live) continue;
        const GroupScale gs = group_scale(m);
        if (t == 0) store_global(dbg, scale + r * lds, gs.scale);
        int8_t *o = q + r * ldq;
        auto store = [&](int k, float4 f) {
            const uint32_t w = quant4(f, gs);
            if constexpr (VEC) {
                const int c = 4 * T * k + 4 * t;
                if (c < cols) store_global(dbg, reinterpret_cast<uint32_t *>(o + c), w);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = 4 * T * k + T * j + t;
                    if (c < cols) store_global(dbg, o + c, int8_t(w >> (8 * j)));
                }
            }
        };
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (k < steps) store(k, v[k]);
        for (int k = KEEP; k < steps; ++k) store(k, load(k));
    }
}

// A CTA takes four units a thread of a row (a unit: four columns with aligned
// rows, else one), all in flight together; the grid's y runs along rows.  Short
// rows get short CTAs (row_threads).
template <int TY, bool VEC>
__global__ void __launch_bounds__(256)
dequantize_kernel(int64_t rows, int cols, const int8_t *__restrict__ q, int64_t ldq,
                  const float *__restrict__ scale, int64_t lds, int shift, void *__restrict__ x, int64_t ldx, DbgAccess dbg) {
    const int units = VEC ? cols / 4 : cols;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const int8_t *qr = q + r * ldq;
        const float *sr = scale + r * lds;
        const int S = blockDim.x;
        for (int64_t i0 = blockIdx.x * int64_t(4 * S) + threadIdx.x; i0 < units; i0 += int64_t(gridDim.x) * 4 * S) {
            uint32_t w[4];
            float s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t i = i0 + S * j < units ? i0 + S * j : 0;
                w[j] = VEC ? load_once(dbg, reinterpret_cast<const uint32_t *>(qr) + i)
                           : uint32_t(uint8_t(load_const(dbg, qr + i)));
                s[j] = load_const(dbg, sr + ((VEC ? 4 * i : i) >> shift));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t i = i0 + S * j;
                if (i >= units) continue;
                if constexpr (VEC) store_four<TY>(dbg, x, r * ldx + 4 * i, unpack_q4(w[j], s[j]));
                else store_one<TY>(dbg, x, r * ldx + i, unpack_q1(int8_t(w[j]), s[j]));
            }
        }
    }
}

struct SwigluArgs : DbgAccess {
    int64_t rows, cols;
    const int8_t *g, *u;
    int64_t ldg, ldu;
    const float *gs, *us;
    int64_t ldgs, ldus;
    int shift;
    const float *dh;
    int64_t lddh;
    float *dg, *du, *h;
    int64_t lddg, lddu, ldh;
};

// Four values of a row from column c on: consecutive with aligned rows (VEC),
// else a CTA's threads apart (so that neighbouring threads hold neighbouring
// columns); past the row's end column 0 is read (no branch: the loads are in
// flight together) and nothing is stored.
template <bool VEC>
__device__ __forceinline__ float4 four_q8(const DbgAccess &d, const int8_t *q, const float *s, int shift, int c, int n) {
    if constexpr (VEC) {
        return unpack_q4(load_once(d, reinterpret_cast<const uint32_t *>(q + c)), load_const(d, s + (c >> shift)));
    } else {
        float v[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int i = c + int(blockDim.x) * t < n ? c + int(blockDim.x) * t : 0;
            v[t] = unpack_q1(load_const(d, q + i), load_const(d, s + (i >> shift)));
        }
        return make_float4(v[0], v[1], v[2], v[3]);
    }
}

template <bool VEC>
__device__ __forceinline__ float4 four_f32(const DbgAccess &d, const float *p, int c, int n) {
    if constexpr (VEC) return load_global(d, reinterpret_cast<const float4 *>(p + c));
    const int S = blockDim.x;
    return make_float4(load_global(d, p + (c < n ? c : 0)), load_global(d, p + (c + S < n ? c + S : 0)),
                       load_global(d, p + (c + 2 * S < n ? c + 2 * S : 0)), load_global(d, p + (c + 3 * S < n ? c + 3 * S : 0)));
}

template <bool VEC>
__device__ __forceinline__ void store_four_f32(const DbgAccess &d, float *p, int c, int n, float4 v) {
    if constexpr (VEC) {
        store_global(d, reinterpret_cast<float4 *>(p + c), v);
    } else {
        const int S = blockDim.x;
        if (c < n) store_global(d, p + c, v.x);
        if (c + S < n) store_global(d, p + c + S, v.y);
        if (c + 2 * S < n) store_global(d, p + c + 2 * S, v.z);
        if (c + 3 * S < n) store_global(d, p + c + 3 * S, v.w);
    }
}

// The backward of h = SiLU(g) * u with g and u restored in registers, the
// operations of swiglu_backward_kernel; with h, the forward's value as well
// (the activation a weight gradient needs, so that it is not kept).  A CTA takes
// four columns a thread of a row.
template <bool VEC, bool H>
__global__ void __launch_bounds__(256) swiglu_backward_i8_kernel(SwigluArgs p) {
    const int n = int(p.cols);
    for (int64_t r = blockIdx.y; r < p.rows; r += gridDim.y) {
        const int8_t *gr = p.g + r * p.ldg, *ur = p.u + r * p.ldu;
        const float *gsr = p.gs + r * p.ldgs, *usr = p.us + r * p.ldus, *dr = p.dh + r * p.lddh;
        float *dgr = p.dg + r * p.lddg, *dur = p.du + r * p.lddu, *hr = H ? p.h + r * p.ldh : nullptr;
        for (int c0 = blockIdx.x * blockDim.x * 4; c0 < n; c0 += gridDim.x * blockDim.x * 4) {
            const int c = c0 + (VEC ? 4 : 1) * threadIdx.x;
            if (c >= n) continue;
            const float4 d = four_f32<VEC>(p, dr, c, n);
            const float4 a = four_q8<VEC>(p, gr, gsr, p.shift, c, n), b = four_q8<VEC>(p, ur, usr, p.shift, c, n);
            float4 og, ou;
            const float2 s01 = sigmoid_fixed2(a.x, a.y), s23 = sigmoid_fixed2(a.z, a.w);
            swiglu_grad_s(a.x, b.x, d.x, s01.x, og.x, ou.x);
            swiglu_grad_s(a.y, b.y, d.y, s01.y, og.y, ou.y);
            swiglu_grad_s(a.z, b.z, d.z, s23.x, og.z, ou.z);
            swiglu_grad_s(a.w, b.w, d.w, s23.y, og.w, ou.w);
            store_four_f32<VEC>(p, dgr, c, n, og);
            store_four_f32<VEC>(p, dur, c, n, ou);
            if constexpr (H)
                store_four_f32<VEC>(p, hr, c, n, make_float4(swiglu_s(a.x, b.x, s01.x), swiglu_s(a.y, b.y, s01.y),
                                                             swiglu_s(a.z, b.z, s23.x), swiglu_s(a.w, b.w, s23.y)));
        }
    }
}

// ------------------------------------------------------------------- host ----

bool aligned(const void *p, int64_t ld, unsigned size, unsigned bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && uint64_t(ld) * size % bytes == 0;
}

// Threads of a CTA that takes four of `units` a thread: whole warps, at most 256.
unsigned row_threads(int64_t units) { return unsigned(std::min<int64_t>(256, ((units + 3) / 4 + 31) / 32 * 32)); }

int sm_count() {
    DeviceInfo di;
    return current_device_info(&di) == REPOPS_OK ? di.sms : 152;
}

template <int TY>
int launch_quantize(int64_t rows, int cols, const void *x, int64_t ldx, int64_t group, int8_t *q, int64_t ldq,
                    float *scale, int64_t lds, const DbgAccess &dbg, cudaStream_t s) {
    const bool vec = cols % 4 == 0 && aligned(x, ldx, storage_size(TY), 4 * storage_size(TY)) && aligned(q, ldq, 1, 4);
    if (group > 0) {
        const int64_t items = rows * ((int64_t(cols) + 511) / 512);
        const unsigned grid = unsigned(std::min<int64_t>((items + 7) / 8, int64_t(sm_count()) * 32));
        if (vec)
            quantize_groups_kernel<TY, true><<<grid, 256, 0, s>>>(rows, cols, x, ldx, int(group), q, ldq, scale, lds, dbg);
        else
            quantize_groups_kernel<TY, false><<<grid, 256, 0, s>>>(rows, cols, x, ldx, int(group), q, ldq, scale, lds, dbg);
        return check_launch();
    }
    // as few threads a row as hold it in registers
    auto go = [&](auto kv, auto ks, int T) {
        const unsigned grid = unsigned(std::min<int64_t>((rows + 256 / T - 1) / (256 / T), int64_t(sm_count()) * 32));
        if (vec) kv<<<grid, 256, 0, s>>>(rows, cols, x, ldx, q, ldq, scale, lds, dbg);
        else ks<<<grid, 256, 0, s>>>(rows, cols, x, ldx, q, ldq, scale, lds, dbg);
        return check_launch();
    };
    if (cols <= 1024) return go(quantize_rows_kernel<TY, true, 32>, quantize_rows_kernel<TY, false, 32>, 32);
    if (cols <= 2048) return go(quantize_rows_kernel<TY, true, 64>, quantize_rows_kernel<TY, false, 64>, 64);
    if (cols <= 4096) return go(quantize_rows_kernel<TY, true, 128>, quantize_rows_kernel<TY, false, 128>, 128);
    return go(quantize_rows_kernel<TY, true, 256>, quantize_rows_kernel<TY, false, 256>, 256);
}

template <int TY>
int launch_dequantize(int64_t rows, int cols, const int8_t *q, int64_t ldq, const float *scale, int64_t lds, int shift,
                      void *x, int64_t ldx, const DbgAccess &dbg, cudaStream_t s) {
    const bool vec = cols % 4 == 0 && aligned(x, ldx, storage_size(TY), 4 * storage_size(TY)) && aligned(q, ldq, 1, 4);
    const int64_t units = vec ? cols / 4 : cols;
    const unsigned threads = row_threads(units);
    const dim3 grid(unsigned((units + 4 * threads - 1) / (4 * threads)), unsigned(std::min<int64_t>(rows, 65535)));
    if (vec) dequantize_kernel<TY, true><<<grid, threads, 0, s>>>(rows, cols, q, ldq, scale, lds, shift, x, ldx, dbg);
    else dequantize_kernel<TY, false><<<grid, threads, 0, s>>>(rows, cols, q, ldq, scale, lds, shift, x, ldx, dbg);
    return check_launch();
}

}  // namespace
}  // namespace repops

using namespace repops;

extern "C" int repops_quantize_rows_i8(int64_t rows, int64_t cols, const void *x, int x_type, int64_t ldx,
                                       int64_t group, int8_t *q, int64_t ldq, float *scale, int64_t lds,
                                       cudaStream_t stream) {
    if (rows < 0 || cols < 0 || cols > (int64_t(1) << 30) || !known_storage(x_type) || !known_group(group))
        return REPOPS_ERR_INVALID_ARG;
    // a row without columns still has its scale where it has one for the row
    if (rows == 0 || group_count(cols, group) == 0) return REPOPS_OK;
    if ((cols > 0 && (!x || !q)) || !scale) return REPOPS_ERR_INVALID_ARG;
    uint64_t xb, qb, sb;
    if (!span_bytes(rows, cols, ldx, storage_size(x_type), &xb) || !span_bytes(rows, cols, ldq, 1, &qb) ||
        !span_bytes(rows, group_count(cols, group), lds, 4, &sb))
        return REPOPS_ERR_INVALID_ARG;
    if (ranges_overlap(q, qb, x, xb) || ranges_overlap(scale, sb, x, xb) || ranges_overlap(q, qb, scale, sb))
        return REPOPS_ERR_ALIAS;
    DbgAccess dbg;
    dbg.reads(x, xb);
    dbg.writes(q, qb);
    dbg.writes(scale, sb);
    if (const int rc = dbg.arm(); rc != REPOPS_OK) return rc;
    switch (x_type) {
        case REPOPS_TYPE_F32:
            return launch_quantize<REPOPS_TYPE_F32>(rows, int(cols), x, ldx, group, q, ldq, scale, lds, dbg, stream);
        case REPOPS_TYPE_F16:
            return launch_quantize<REPOPS_TYPE_F16>(rows, int(cols), x, ldx, group, q, ldq, scale, lds, dbg, stream);
        default:
            return launch_quantize<REPOPS_TYPE_BF16>(rows, int(cols), x, ldx, group, q, ldq, scale, lds, dbg, stream);
    }
}

extern "C" int repops_dequantize_rows_i8(int64_t rows, int64_t cols, const int8_t *q, int64_t ldq,
                                         const float *scale, int64_t lds, int64_t group, void *x, int x_type,
                                         int64_t ldx, cudaStream_t stream) {
    if (rows < 0 || cols < 0 || cols > (int64_t(1) << 30) || !known_storage(x_type) || !known_group(group))
        return REPOPS_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return REPOPS_OK;
    if (!x || !q || !scale) return REPOPS_ERR_INVALID_ARG;
    uint64_t xb, qb, sb;
    if (!span_bytes(rows, cols, ldx, storage_size(x_type), &xb) || !span_bytes(rows, cols, ldq, 1, &qb) ||
        !span_bytes(rows, group_count(cols, group), lds, 4, &sb))
        return REPOPS_ERR_INVALID_ARG;
    if (ranges_overlap(x, xb, q, qb) || ranges_overlap(x, xb, scale, sb)) return REPOPS_ERR_ALIAS;
    const int shift = group_shift(group);
    DbgAccess dbg;
    dbg.reads(q, qb);
    dbg.reads(scale, sb);
    dbg.writes(x, xb);
    if (const int rc = dbg.arm(); rc != REPOPS_OK) return rc;
    switch (x_type) {
        case REPOPS_TYPE_F32:
            return launch_dequantize<REPOPS_TYPE_F32>(rows, int(cols), q, ldq, scale, lds, shift, x, ldx, dbg, stream);
        case REPOPS_TYPE_F16:
            return launch_dequantize<REPOPS_TYPE_F16>(rows, int(cols), q, ldq, scale, lds, shift, x, ldx, dbg, stream);
        default:
            return launch_dequantize<REPOPS_TYPE_BF16>(rows, int(cols), q, ldq, scale, lds, shift, x, ldx, dbg, stream);
    }
}

extern "C" int repops_swiglu_backward_i8(int64_t rows, int64_t cols, const int8_t *g, int64_t ldg,
                                         const float *g_scale, int64_t ldgs, const int8_t *u, int64_t ldu,
                                         const float *u_scale, int64_t ldus, int64_t group, const float *dh,
                                         int64_t lddh, float *dg, int64_t lddg, float *du, int64_t lddu, float *h,
                                         int64_t ldh, cudaStream_t stream) {
    if (rows < 0 || cols < 0 || cols > (int64_t(1) << 30) || !known_group(group)) return REPOPS_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return REPOPS_OK;
    if (!g || !g_scale || !u || !u_scale || !dh || !dg || !du) return REPOPS_ERR_INVALID_ARG;
    const int64_t ng = group_count(cols, group);
    uint64_t gb, gsb, ub, usb, db, ogb, oub, hb = 0;
    if (!span_bytes(rows, cols, ldg, 1, &gb) || !span_bytes(rows, ng, ldgs, 4, &gsb) ||
        !span_bytes(rows, cols, ldu, 1, &ub) || !span_bytes(rows, ng, ldus, 4, &usb) ||
        !span_bytes(rows, cols, lddh, 4, &db) || !span_bytes(rows, cols, lddg, 4, &ogb) ||
        !span_bytes(rows, cols, lddu, 4, &oub) || (h && !span_bytes(rows, cols, ldh, 4, &hb)))
        return REPOPS_ERR_INVALID_ARG;
    // every output apart from the inputs, and (as column blocks of one matrix
    // may interleave) no element of one output another's; one of them may be
    // dh itself, each element being read before it is written
    const struct { float *p; uint64_t b; int64_t ld; } outs[3] = {{dg, ogb, lddg}, {du, oub, lddu}, {h, hb, ldh}};
    for (int i = 0; i < 3; ++i) {
        if (!outs[i].p) continue;
        if (ranges_overlap(outs[i].p, outs[i].b, g, gb) || ranges_overlap(outs[i].p, outs[i].b, g_scale, gsb) ||
            ranges_overlap(outs[i].p, outs[i].b, u, ub) || ranges_overlap(outs[i].p, outs[i].b, u_scale, usb))
            return REPOPS_ERR_ALIAS;
        if (bad_overlap(outs[i].p, outs[i].ld, dh, lddh, rows, cols)) return REPOPS_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (outs[j].p && blocks_overlap(outs[i].p, outs[i].ld, outs[j].p, outs[j].ld, rows, cols))
                return REPOPS_ERR_ALIAS;
    }
    SwigluArgs a{{}, rows, cols, g, u, ldg, ldu, g_scale, u_scale, ldgs, ldus, group_shift(group), dh, lddh,
                 dg, du, h, lddg, lddu, ldh};
    a.reads(g, gb);
    a.reads(u, ub);
    a.reads(g_scale, gsb);
    a.reads(u_scale, usb);
    a.reads(dh, db);
    a.writes(dg, ogb);
    a.writes(du, oub);
    a.writes(h, hb);
    if (const int rc = a.arm(); rc != REPOPS_OK) return rc;
    const bool vec = cols % 4 == 0 && aligned(g, ldg, 1, 4) && aligned(u, ldu, 1, 4) && aligned(dh, lddh, 4, 16) &&
                     aligned(dg, lddg, 4, 16) && aligned(du, lddu, 4, 16) && (!h || aligned(h, ldh, 4, 16));
    const unsigned threads = row_threads(cols);
    const dim3 grid(unsigned((cols + 4 * threads - 1) / (4 * threads)), unsigned(std::min<int64_t>(rows, 65535)));
    if (vec && h) swiglu_backward_i8_kernel<true, true><<<grid, threads, 0, stream>>>(a);
    else if (vec) swiglu_backward_i8_kernel<true, false><<<grid, threads, 0, stream>>>(a);
    else if (h) swiglu_backward_i8_kernel<false, true><<<grid, threads, 0, stream>>>(a);
    else swiglu_backward_i8_kernel<false, false><<<grid, threads, 0, stream>>>(a);
    return check_launch();
}
