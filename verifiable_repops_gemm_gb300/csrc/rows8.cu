// rows8.cu -- activations kept in 8 bits: rows quantised with a scale for each
// group of columns, restored, and SwiGLU's backward read straight from them.
//
// Format, for every group of a row, each step one binary32 rounding:
//   amax = max |x|,  a = max(amax, 2^-100),
//   scale = fl(a / 127),  q = rint(fl(x * fl(127 / a))) (ties to even);
// |x| <= a, so fl(x * fl(127 / a)) <= 127 * (1 + 2^-23) and rint gives at most
// 127: no clamp.  The floor keeps 127 / a finite: a group below it becomes
// zeros, an error of at most 2^-100.  A group holding an infinity or a NaN gets
// scale NaN and q = 0, so it comes back as NaN instead of as wrong numbers.
// The maximum does not depend on the order it is taken in, so neither does any
// bit here.
//
// All kernels stream: they are bound by memory.  Bytes an element: quantising
// 4 (or 2) + 1, restoring 1 + 4, the backward 2 + 4 in and 12 out.
#include <algorithm>

#include "internal.cuh"
#include "rows8.cuh"
#include "swiglu.cuh"

namespace repops {
namespace {

constexpr float kScaleFloor = 0x1p-100f;

template <int TY>
__device__ __forceinline__ float load_one(const void *p, int64_t i) {
    if constexpr (TY == REPOPS_TYPE_F32) return static_cast<const float *>(p)[i];
    else if constexpr (TY == REPOPS_TYPE_F16) return __half2float(static_cast<const __half *>(p)[i]);
    else return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

template <int TY>
__device__ __forceinline__ void store_one(void *p, int64_t i, float v) {
    if constexpr (TY == REPOPS_TYPE_F32) static_cast<float *>(p)[i] = v;
    else if constexpr (TY == REPOPS_TYPE_F16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// Elements i .. i+3, i a multiple of 4 elements from an aligned base.
template <int TY>
__device__ __forceinline__ float4 load_four(const void *p, int64_t i) {
    if constexpr (TY == REPOPS_TYPE_F32) {
        return __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
    } else {
        const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i));
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
__device__ __forceinline__ void store_four(void *p, int64_t i, float4 v) {
    if constexpr (TY == REPOPS_TYPE_F32) {
        __stcs(reinterpret_cast<float4 *>(static_cast<float *>(p) + i), v);
    } else {
        uint16_t h[4];
        store_one<TY>(h, 0, v.x);
        store_one<TY>(h, 1, v.y);
        store_one<TY>(h, 2, v.z);
        store_one<TY>(h, 3, v.w);
        __stcs(reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i),
               make_uint2(h[0] | (unsigned(h[1]) << 16), h[2] | (unsigned(h[3]) << 16)));
    }
}

// The larger magnitude, a NaN winning over everything: magnitudes are compared
// as their bit patterns, which order non-negative values, infinity and NaN.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t mag4(uint32_t m, float4 v) {
    return max(max(max(mag(v.x), mag(v.y)), max(mag(v.z), mag(v.w))), m);
}

struct GroupScale {
    float scale, inv;
};

__device__ __forceinline__ GroupScale group_scale(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return {__uint_as_float(0x7fffffffu), 0.0f};
    const float a = fmaxf(__uint_as_float(amax_bits), kScaleFloor);
    return {__fdiv_rn(a, 127.0f), __fdiv_rn(127.0f, a)};
}

// A non-finite group has inv 0: its q is 0 for the finite values, and for the
// others (inf * 0 = NaN) the conversion of NaN, which is 0 as well.
__device__ __forceinline__ int quant1(float x, float inv) { return __float2int_rn(__fmul_rn(x, inv)); }

__device__ __forceinline__ uint32_t quant4(float4 v, float inv) {
    return (uint32_t(quant1(v.x, inv)) & 0xffu) | ((uint32_t(quant1(v.y, inv)) & 0xffu) << 8) |
           ((uint32_t(quant1(v.z, inv)) & 0xffu) << 16) | (uint32_t(quant1(v.w, inv)) << 24);
}

// Groups of 32 .. 256 columns: a warp takes 256 columns of a row as two loads
// of four values a lane (columns 4*lane and 128 + 4*lane), so a group is 8, 16
// or 32 lanes of one load, or both loads: its maximum is 3 to 5 shuffles.
template <int TY, bool VEC>
__global__ void __launch_bounds__(256)
quantize_groups_kernel(int64_t rows, int64_t cols, const void *__restrict__ x, int64_t ldx, int group,
                       int8_t *__restrict__ q, int64_t ldq, float *__restrict__ scale, int64_t lds) {
    const int lane = threadIdx.x & 31;
    const int64_t segs = (cols + 255) / 256;
    const int64_t items = rows * segs, stride = int64_t(gridDim.x) * 8;
    const int width = min(group, 128) / 4;          // lanes of a group within one load
    for (int64_t it = blockIdx.x * int64_t(8) + (threadIdx.x >> 5); it < items; it += stride) {
        const int64_t r = it / segs, c0 = (it - r * segs) * 256 + 4 * lane;
        float4 v[2];
        uint32_t m[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int64_t c = c0 + 128 * s, base = r * ldx + c;
            if constexpr (VEC) {
                v[s] = c < cols ? load_four<TY>(x, base) : make_float4(0.f, 0.f, 0.f, 0.f);
            } else {
                v[s].x = c < cols ? load_one<TY>(x, base) : 0.0f;
                v[s].y = c + 1 < cols ? load_one<TY>(x, base + 1) : 0.0f;
                v[s].z = c + 2 < cols ? load_one<TY>(x, base + 2) : 0.0f;
                v[s].w = c + 3 < cols ? load_one<TY>(x, base + 3) : 0.0f;
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) m[s] = mag4(0u, v[s]);
        if (group == 256) m[0] = m[1] = max(m[0], m[1]);
        for (int o = width / 2; o > 0; o >>= 1) {
            m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
            m[1] = max(m[1], __shfl_xor_sync(0xffffffffu, m[1], o));
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int64_t c = c0 + 128 * s;
            if (c >= cols) continue;
            const GroupScale gs = group_scale(m[s]);
            const uint32_t w = quant4(v[s], gs.inv);
            int8_t *o = q + r * ldq + c;
            if constexpr (VEC) {
                __stcs(reinterpret_cast<uint32_t *>(o), w);
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (c + t < cols) o[t] = int8_t(w >> (8 * t));
            }
            if (c % group == 0) scale[r * lds + c / group] = gs.scale;
        }
    }
}

// One scale a row: T threads a row (a warp, or the CTA), each keeping up to
// 4 * KEEP of the row's values in registers between the maximum and the
// quantisation; longer rows are read again from the cache.
template <int TY, bool VEC, int T>
__global__ void __launch_bounds__(256)
quantize_rows_kernel(int64_t rows, int64_t cols, const void *__restrict__ x, int64_t ldx, int8_t *__restrict__ q,
                     int64_t ldq, float *__restrict__ scale, int64_t lds) {
    constexpr int KEEP = 8, ROWS = 256 / T, STEP = VEC ? 4 * T : T;
    __shared__ uint32_t part[8];
    const int t = threadIdx.x % T;
    for (int64_t r0 = blockIdx.x * int64_t(ROWS); r0 < rows; r0 += int64_t(gridDim.x) * ROWS) {
        const int64_t r = r0 + threadIdx.x / T;
        const bool live = r < rows;
        const int64_t base = r * ldx;
        // step k covers columns [k * STEP, (k + 1) * STEP): VEC four a thread,
        // else one a thread (four steps make one float4 here)
        float4 v[KEEP];
        auto load = [&](int64_t k) {
            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
            if constexpr (VEC) {
                const int64_t c = k * STEP + 4 * t;
                if (c < cols) w = load_four<TY>(x, base + c);
            } else {
                const int64_t c = 4 * k * STEP + t;
                if (c < cols) w.x = load_one<TY>(x, base + c);
                if (c + STEP < cols) w.y = load_one<TY>(x, base + c + STEP);
                if (c + 2 * STEP < cols) w.z = load_one<TY>(x, base + c + 2 * STEP);
                if (c + 3 * STEP < cols) w.w = load_one<TY>(x, base + c + 3 * STEP);
            }
            return w;
        };
        const int64_t steps = (cols + 4 * T - 1) / (4 * T);
        uint32_t m = 0;
        if (live) {
#pragma unroll
            for (int k = 0; k < KEEP; ++k)
                if (k < steps) v[k] = load(k);
#pragma unroll
            for (int k = 0; k < KEEP; ++k)
                if (k < steps) m = mag4(m, v[k]);
            for (int64_t k = KEEP; k < steps; ++k) m = mag4(m, load(k));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if constexpr (T > 32) {
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < T / 32; ++w) m = max(m, part[w]);
            __syncthreads();
        }
        if (!live) continue;
        const GroupScale gs = group_scale(m);
        if (t == 0) scale[r * lds] = gs.scale;
        int8_t *o = q + r * ldq;
        auto store = [&](int64_t k, float4 f) {
            const uint32_t w = quant4(f, gs.inv);
            if constexpr (VEC) {
                const int64_t c = k * STEP + 4 * t;
                if (c < cols) *reinterpret_cast<uint32_t *>(o + c) = w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t c = (4 * k + j) * STEP + t;
                    if (c < cols) o[c] = int8_t(w >> (8 * j));
                }
            }
        };
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (k < steps) store(k, v[k]);
        for (int64_t k = KEEP; k < steps; ++k) store(k, load(k));
    }
}

// Threads along columns (four each, or one), the grid's y along rows.
template <int TY, bool VEC>
__global__ void __launch_bounds__(256)
dequantize_kernel(int64_t rows, int64_t cols, const int8_t *__restrict__ q, int64_t ldq,
                  const float *__restrict__ scale, int64_t lds, int shift, void *__restrict__ x, int64_t ldx) {
    const int64_t units = VEC ? cols / 4 : cols;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const int8_t *qr = q + r * ldq;
        const float *sr = scale + r * lds;
        for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < units;
             i += int64_t(gridDim.x) * blockDim.x) {
            if constexpr (VEC) {
                const uint32_t w = __ldcs(reinterpret_cast<const uint32_t *>(qr) + i);
                store_four<TY>(x, r * ldx + 4 * i, unpack_q4(w, __ldg(sr + ((4 * i) >> shift))));
            } else {
                store_one<TY>(x, r * ldx + i, __fmul_rn(float(qr[i]), __ldg(sr + (i >> shift))));
            }
        }
    }
}

struct SwigluArgs {
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

// The backward of h = SiLU(g) * u with g and u restored in registers, the
// operations of swiglu_backward_kernel; with h, the forward's value as well
// (the activation a weight gradient needs, so that it is not kept).
template <bool VEC, bool H>
__global__ void __launch_bounds__(256) swiglu_backward_i8_kernel(SwigluArgs p) {
    const int64_t units = VEC ? p.cols / 4 : p.cols;
    for (int64_t r = blockIdx.y; r < p.rows; r += gridDim.y) {
        const int8_t *gr = p.g + r * p.ldg, *ur = p.u + r * p.ldu;
        const float *gsr = p.gs + r * p.ldgs, *usr = p.us + r * p.ldus, *dr = p.dh + r * p.lddh;
        float *dgr = p.dg + r * p.lddg, *dur = p.du + r * p.lddu, *hr = H ? p.h + r * p.ldh : nullptr;
        for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < units;
             i += int64_t(gridDim.x) * blockDim.x) {
            if constexpr (VEC) {
                const int64_t grp = (4 * i) >> p.shift;
                const float4 d = reinterpret_cast<const float4 *>(dr)[i];
                const float4 a = unpack_q4(__ldcs(reinterpret_cast<const uint32_t *>(gr) + i), __ldg(gsr + grp));
                const float4 b = unpack_q4(__ldcs(reinterpret_cast<const uint32_t *>(ur) + i), __ldg(usr + grp));
                float4 og, ou;
                const float2 s01 = sigmoid_fixed2(a.x, a.y), s23 = sigmoid_fixed2(a.z, a.w);
                swiglu_grad_s(a.x, b.x, d.x, s01.x, og.x, ou.x);
                swiglu_grad_s(a.y, b.y, d.y, s01.y, og.y, ou.y);
                swiglu_grad_s(a.z, b.z, d.z, s23.x, og.z, ou.z);
                swiglu_grad_s(a.w, b.w, d.w, s23.y, og.w, ou.w);
                reinterpret_cast<float4 *>(dgr)[i] = og;
                reinterpret_cast<float4 *>(dur)[i] = ou;
                if constexpr (H)
                    reinterpret_cast<float4 *>(hr)[i] =
                        make_float4(swiglu_s(a.x, b.x, s01.x), swiglu_s(a.y, b.y, s01.y),
                                    swiglu_s(a.z, b.z, s23.x), swiglu_s(a.w, b.w, s23.y));
            } else {
                const int64_t grp = i >> p.shift;
                const float a = __fmul_rn(float(gr[i]), __ldg(gsr + grp));
                const float b = __fmul_rn(float(ur[i]), __ldg(usr + grp));
                float og, ou;
                const float d = dr[i];
                swiglu_grad1(a, b, d, og, ou);
                dgr[i] = og;
                dur[i] = ou;
                if constexpr (H) hr[i] = swiglu1(a, b);
            }
        }
    }
}

// ------------------------------------------------------------------- host ----

bool aligned(const void *p, int64_t ld, unsigned size, unsigned bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && uint64_t(ld) * size % bytes == 0;
}

int sm_count() {
    DeviceInfo di;
    return current_device_info(&di) == REPOPS_OK ? di.sms : 152;
}

// 256-thread CTAs: x over column units, y over rows, about 16 CTAs per SM.
dim3 grid_2d(int64_t units, int64_t rows) {
    const int64_t target = int64_t(sm_count()) * 16;
    const int64_t gx = std::max<int64_t>(1, std::min<int64_t>((units + 255) / 256, target));
    const int64_t gy = std::max<int64_t>(1, std::min<int64_t>({rows, std::max<int64_t>(1, target / gx), 65535}));
    return dim3(unsigned(gx), unsigned(gy));
}

template <int TY>
int launch_quantize(int64_t rows, int64_t cols, const void *x, int64_t ldx, int64_t group, int8_t *q, int64_t ldq,
                    float *scale, int64_t lds, cudaStream_t s) {
    const bool vec = cols % 4 == 0 && aligned(x, ldx, storage_size(TY), 4 * storage_size(TY)) && aligned(q, ldq, 1, 4);
    if (group > 0) {
        const int64_t items = rows * ((cols + 255) / 256);
        const unsigned grid = unsigned(std::min<int64_t>((items + 7) / 8, int64_t(sm_count()) * 32));
        if (vec)
            quantize_groups_kernel<TY, true><<<grid, 256, 0, s>>>(rows, cols, x, ldx, int(group), q, ldq, scale, lds);
        else
            quantize_groups_kernel<TY, false><<<grid, 256, 0, s>>>(rows, cols, x, ldx, int(group), q, ldq, scale, lds);
        return check_launch();
    }
    // a warp a row while the row fits its registers, else the CTA
    const bool warp = cols <= 1024;
    const unsigned grid = unsigned(std::min<int64_t>(warp ? (rows + 7) / 8 : rows, int64_t(sm_count()) * 32));
    if (warp && vec)
        quantize_rows_kernel<TY, true, 32><<<grid, 256, 0, s>>>(rows, cols, x, ldx, q, ldq, scale, lds);
    else if (warp)
        quantize_rows_kernel<TY, false, 32><<<grid, 256, 0, s>>>(rows, cols, x, ldx, q, ldq, scale, lds);
    else if (vec)
        quantize_rows_kernel<TY, true, 256><<<grid, 256, 0, s>>>(rows, cols, x, ldx, q, ldq, scale, lds);
    else
        quantize_rows_kernel<TY, false, 256><<<grid, 256, 0, s>>>(rows, cols, x, ldx, q, ldq, scale, lds);
    return check_launch();
}

template <int TY>
int launch_dequantize(int64_t rows, int64_t cols, const int8_t *q, int64_t ldq, const float *scale, int64_t lds,
                      int shift, void *x, int64_t ldx, cudaStream_t s) {
    const bool vec = cols % 4 == 0 && aligned(x, ldx, storage_size(TY), 4 * storage_size(TY)) && aligned(q, ldq, 1, 4);
    if (vec)
        dequantize_kernel<TY, true><<<grid_2d(cols / 4, rows), 256, 0, s>>>(rows, cols, q, ldq, scale, lds, shift, x, ldx);
    else
        dequantize_kernel<TY, false><<<grid_2d(cols, rows), 256, 0, s>>>(rows, cols, q, ldq, scale, lds, shift, x, ldx);
    return check_launch();
}

}  // namespace
}  // namespace repops

using namespace repops;

extern "C" int repops_quantize_rows_i8(int64_t rows, int64_t cols, const void *x, int x_type, int64_t ldx,
                                       int64_t group, int8_t *q, int64_t ldq, float *scale, int64_t lds,
                                       cudaStream_t stream) {
    if (rows < 0 || cols < 0 || cols > INT32_MAX || !known_storage(x_type) || !known_group(group))
        return REPOPS_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return REPOPS_OK;
    if (!x || !q || !scale) return REPOPS_ERR_INVALID_ARG;
    uint64_t xb, qb, sb;
    if (!span_bytes(rows, cols, ldx, storage_size(x_type), &xb) || !span_bytes(rows, cols, ldq, 1, &qb) ||
        !span_bytes(rows, group_count(cols, group), lds, 4, &sb))
        return REPOPS_ERR_INVALID_ARG;
    if (ranges_overlap(q, qb, x, xb) || ranges_overlap(scale, sb, x, xb) || ranges_overlap(q, qb, scale, sb))
        return REPOPS_ERR_ALIAS;
    switch (x_type) {
        case REPOPS_TYPE_F32:
            return launch_quantize<REPOPS_TYPE_F32>(rows, cols, x, ldx, group, q, ldq, scale, lds, stream);
        case REPOPS_TYPE_F16:
            return launch_quantize<REPOPS_TYPE_F16>(rows, cols, x, ldx, group, q, ldq, scale, lds, stream);
        default:
            return launch_quantize<REPOPS_TYPE_BF16>(rows, cols, x, ldx, group, q, ldq, scale, lds, stream);
    }
}

extern "C" int repops_dequantize_rows_i8(int64_t rows, int64_t cols, const int8_t *q, int64_t ldq,
                                         const float *scale, int64_t lds, int64_t group, void *x, int x_type,
                                         int64_t ldx, cudaStream_t stream) {
    if (rows < 0 || cols < 0 || cols > INT32_MAX || !known_storage(x_type) || !known_group(group))
        return REPOPS_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return REPOPS_OK;
    if (!x || !q || !scale) return REPOPS_ERR_INVALID_ARG;
    uint64_t xb, qb, sb;
    if (!span_bytes(rows, cols, ldx, storage_size(x_type), &xb) || !span_bytes(rows, cols, ldq, 1, &qb) ||
        !span_bytes(rows, group_count(cols, group), lds, 4, &sb))
        return REPOPS_ERR_INVALID_ARG;
    if (ranges_overlap(x, xb, q, qb) || ranges_overlap(x, xb, scale, sb)) return REPOPS_ERR_ALIAS;
    const int shift = group_shift(group);
    switch (x_type) {
        case REPOPS_TYPE_F32:
            return launch_dequantize<REPOPS_TYPE_F32>(rows, cols, q, ldq, scale, lds, shift, x, ldx, stream);
        case REPOPS_TYPE_F16:
            return launch_dequantize<REPOPS_TYPE_F16>(rows, cols, q, ldq, scale, lds, shift, x, ldx, stream);
        default:
            return launch_dequantize<REPOPS_TYPE_BF16>(rows, cols, q, ldq, scale, lds, shift, x, ldx, stream);
    }
}

extern "C" int repops_swiglu_backward_i8(int64_t rows, int64_t cols, const int8_t *g, int64_t ldg,
                                         const float *g_scale, int64_t ldgs, const int8_t *u, int64_t ldu,
                                         const float *u_scale, int64_t ldus, int64_t group, const float *dh,
                                         int64_t lddh, float *dg, int64_t lddg, float *du, int64_t lddu, float *h,
                                         int64_t ldh, cudaStream_t stream) {
    if (rows < 0 || cols < 0 || cols > INT32_MAX || !known_group(group)) return REPOPS_ERR_INVALID_ARG;
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
    const SwigluArgs a{rows, cols, g, u, ldg, ldu, g_scale, u_scale, ldgs, ldus, group_shift(group), dh, lddh,
                       dg, du, h, lddg, lddu, ldh};
    const bool vec = cols % 4 == 0 && aligned(g, ldg, 1, 4) && aligned(u, ldu, 1, 4) && aligned(dh, lddh, 4, 16) &&
                     aligned(dg, lddg, 4, 16) && aligned(du, lddu, 4, 16) && (!h || aligned(h, ldh, 4, 16));
    const dim3 grid = grid_2d(vec ? cols / 4 : cols, rows);
    if (vec && h) swiglu_backward_i8_kernel<true, true><<<grid, 256, 0, stream>>>(a);
    else if (vec) swiglu_backward_i8_kernel<true, false><<<grid, 256, 0, stream>>>(a);
    else if (h) swiglu_backward_i8_kernel<false, true><<<grid, 256, 0, stream>>>(a);
    else swiglu_backward_i8_kernel<false, false><<<grid, 256, 0, stream>>>(a);
    return check_launch();
}
