// gemm_i8.cu -- matrix product of 8-bit integers with a scale for each row of A
// (token) and each column of B (channel).
//
//   acc[i][j] = sum_k A[i][k] * B[j][k]        (whole numbers, exact)
//   C[i][j]   = narrow(fl(fl(fl(acc) * a_scale[i]) * b_scale[j]) [+ bias[j]])
//
// A sum of whole numbers is the same in every order, so the product needs no
// fixed k-chain: it may be split over k and run on the tensor cores, and still
// every kernel here gives the same bits.  |acc| <= 2^14 * K < 2^31 for K <
// 131072.
//
// Few rows of A (a token being generated, or the tokens of a few sequences):
// bound by reading B once.  The integer tensor instruction (mma.sync
// m16n8k32.s8) takes 16 channels x 8 tokens x 32 k straight from 16-byte global
// loads: which k a lane holds does not matter as long as both operands agree,
// so lane q of a quad loads k = 16q .. 16q + 15 of a 64-k step and feeds words
// 0, 1 to one instruction and 2, 3 to the next.  The warps of a CTA split k and
// add their sums in shared memory.
//
// Many rows: the operands are widened once to binary16 (exact: 8 bits fit its
// 11) and multiplied by tcgen05 with binary32 accumulators in tensor memory,
// because this chip's integer tensor rate is a small part of its binary16 rate.
// Every product and every partial sum of up to 512 of them is a whole number
// below 2^23 in magnitude, so binary32 accumulation is exact whatever its
// order; after each 512 of k the accumulators are added to 32-bit integers in
// registers while the tensor core fills the other half of tensor memory.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gemm_common.h"
#include "internal.cuh"
#include "rows8.cuh"
#include "tcgen05.cuh"

namespace repops {
namespace {

constexpr int64_t kMaxK = 131071;

struct I8Args {
    int64_t M, N, K;
    const int8_t *A, *B;           // M x K and N x K, k contiguous
    int64_t lda, ldb;
    const float *sa, *sb, *bias;   // bias may be null
    void *C;
    int64_t ldc;
    const int8_t *a_end, *b_end;   // one past each operand's last byte
};

// ---------------------------------------------------------- operand bytes ----

// Bytes k .. k+15 of a row (zeros from `n` on), whatever the row's alignment.
// VEC: the row is 16-byte aligned.  Otherwise five aligned words are shifted
// together; where those would leave the operand [base, end), single bytes.
template <bool VEC>
__device__ __forceinline__ uint4 load_k16(const int8_t *__restrict__ row, int64_t k, int64_t n, const int8_t *base,
                                          const int8_t *end) {
    const int8_t *p = row + k;
    if (k + 16 <= n) {
        if constexpr (VEC) {
            return __ldg(reinterpret_cast<const uint4 *>(p));
        } else {
            const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(p) & 3u);
            const int8_t *q = p - off;
            if (q >= base && q + (off ? 20 : 16) <= end) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(q);
                const uint32_t a = __ldg(w), b = __ldg(w + 1), c = __ldg(w + 2), d = __ldg(w + 3),
                               e = off ? __ldg(w + 4) : 0u;
                const uint32_t s = 8 * off;
                return make_uint4(__funnelshift_r(a, b, s), __funnelshift_r(b, c, s), __funnelshift_r(c, d, s),
                                  __funnelshift_r(d, e, s));
            }
        }
    }
    uint32_t r[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (k + i < n) r[i >> 2] |= uint32_t(uint8_t(p[i])) << (8 * (i & 3));
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// ---------------------------------------------------------------- epilogue ----

template <int TY>
__device__ __forceinline__ void store_c(void *C, int64_t i, float v) {
    if constexpr (TY == REPOPS_TYPE_F32) static_cast<float *>(C)[i] = v;
    else if constexpr (TY == REPOPS_TYPE_F16) static_cast<__half *>(C)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(C)[i] = __float2bfloat16_rn(v);
}

template <int TY>
__device__ __forceinline__ uint32_t pack_c(float lo, float hi) {
    uint16_t h[2];
    store_c<TY>(h, 0, lo);
    store_c<TY>(h, 1, hi);
    return h[0] | (uint32_t(h[1]) << 16);
}

__device__ __forceinline__ float scale_bias(float v, float sb, const float *bias, int64_t j) {
    v = __fmul_rn(v, sb);
    return bias ? __fadd_rn(v, __ldg(bias + j)) : v;
}

// ---------------------------------------------------------------- few rows ----

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 * MT channels x 8 * NT tokens a CTA of 8 warps; warp w takes the 64-k
// steps w, w + 8, ...
template <int TY, int MT, int NT, bool VEC>
__global__ void __launch_bounds__(256) gemm_i8_rows_kernel(I8Args p) {
    constexpr int CH = 16 * MT, TK = 8 * NT;
    __shared__ int sum[TK][CH + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int64_t n0 = int64_t(blockIdx.x) * CH, m0 = int64_t(blockIdx.y) * TK;
    for (int i = threadIdx.x; i < TK * (CH + 1); i += 256) (&sum[0][0])[i] = 0;
    int d[MT][NT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) d[t][u][i] = 0;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const int64_t steps = (p.K + 63) / 64;
#pragma unroll 2
    for (int64_t s = warp; s < steps; s += 8) {
        const int64_t k = s * 64 + 16 * q;
        uint4 w[MT][2], x[NT];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t j = n0 + 16 * t + 8 * h + g;
                w[t][h] = j < p.N && k < p.K ? load_k16<VEC>(p.B + j * p.ldb, k, p.K, p.B, p.b_end) : zero;
            }
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const int64_t i = m0 + 8 * u + g;
            x[u] = i < p.M && k < p.K ? load_k16<VEC>(p.A + i * p.lda, k, p.K, p.A, p.a_end) : zero;
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                mma_s8(d[t][u], w[t][0].x, w[t][1].x, w[t][0].y, w[t][1].y, x[u].x, x[u].y);
                mma_s8(d[t][u], w[t][0].z, w[t][1].z, w[t][0].w, w[t][1].w, x[u].z, x[u].w);
            }
    }
    __syncthreads();
    // lane: channels g and g + 8, tokens 2q and 2q + 1 of each tile
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                atomicAdd(&sum[8 * u + 2 * q + (i & 1)][16 * t + 8 * (i >> 1) + g], d[t][u][i]);
    __syncthreads();
    for (int i = threadIdx.x; i < TK * CH; i += 256) {
        const int64_t m = m0 + i / CH, n = n0 + i % CH;
        if (m >= p.M || n >= p.N) continue;
        const float v = __fmul_rn(__int2float_rn(sum[i / CH][i % CH]), __ldg(p.sa + m));
        store_c<TY>(p.C, m * p.ldc + n, scale_bias(v, __ldg(p.sb + n), p.bias, n));
    }
}

// --------------------------------------------------------------- many rows ----

constexpr int BM = 128, BK = 64;          // BK binary16 = one 128-byte swizzled row
constexpr int kChunkSteps = 8;            // k-steps between two drains: 512 of k

// Whole numbers as binary16: with the sign bit flipped a byte is q + 128, the
// low mantissa bits of 1024 + (q + 128); subtracting 1152 is exact.
__device__ __forceinline__ uint32_t widen2(uint32_t w, uint32_t selector) {
    const uint32_t h = __byte_perm(w, 0x64646464u, selector);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&h), __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The rows of A, then those of B, as binary16 rows of Kp (a multiple of 64)
// values, zeros past K: 16 values a thread.
template <bool VEC>
__global__ void __launch_bounds__(256) widen_kernel(I8Args p, int64_t Kp, __half *__restrict__ out) {
    const int64_t per = Kp / 16, items = (p.M + p.N) * per, stride = int64_t(gridDim.x) * 256;
    for (int64_t it = blockIdx.x * int64_t(256) + threadIdx.x; it < items; it += stride) {
        const int64_t r = it / per, k = (it - r * per) * 16;
        const bool a = r < p.M;
        const uint4 w = a ? load_k16<VEC>(p.A + r * p.lda, k, p.K, p.A, p.a_end)
                          : load_k16<VEC>(p.B + (r - p.M) * p.ldb, k, p.K, p.B, p.b_end);
        const uint32_t b[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
        uint4 *o = reinterpret_cast<uint4 *>(out + it * 16);
        o[0] = make_uint4(widen2(b[0], 0x4140u), widen2(b[0], 0x4342u), widen2(b[1], 0x4140u), widen2(b[1], 0x4342u));
        o[1] = make_uint4(widen2(b[2], 0x4140u), widen2(b[2], 0x4342u), widen2(b[3], 0x4140u), widen2(b[3], 0x4342u));
    }
}

template <int BN>
struct TileCfg {
    static constexpr int STAGE_BYTES = (BM + BN) * BK * 2;
    static constexpr int STAGES = 196608 / STAGE_BYTES;          // 4, 6 or 8
    static constexpr int WARP_STAGE = 32 * 32 * 4;               // an epilogue warp's 32 x 32 block
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + 8 * WARP_STAGE;
    static constexpr uint32_t TMEM_COLS = 2 * BN;
    static constexpr int COLS = BN / 2;                          // an epilogue warp's columns
};

constexpr int kTileThreads = 320;         // 8 epilogue warps, a TMA warp, an MMA warp

struct TileMap {
    int tiles_m, tiles_n, band;           // band: tile rows walked together, for L2 reuse
    __device__ __forceinline__ void at(int t, int &m, int &n) const {
        const int per = band * tiles_n, b = t / per, first = b * band, rows = min(band, tiles_m - first);
        const int r = t - b * per;
        n = r / rows;
        m = first + r - n * rows;
    }
};

template <int TY, int BN>
__global__ void __launch_bounds__(kTileThreads, 1)
gemm_i8_tile_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, I8Args p,
                    TileMap tm, int ksteps, int c_vec, unsigned *status) {
    using T = TileCfg<BN>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[T::STAGES], empty[T::STAGES], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_slot;
    uint8_t *stages = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = tm.tiles_m * tm.tiles_n;
    const int chunks = (ksteps + kChunkSteps - 1) / kChunkSteps;
    if (threadIdx.x == 0) {
        for (int s = 0; s < T::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);
        }
        mbar_init(&drained, 1);
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc(&tmem_slot, T::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // Every wait gives up after its limit: the role that gave up sets the
    // status word, waits (again with a limit) for its own copies or products in
    // flight and leaves; the others run into their own limits.
    if (warp == 8) {
        if (lane == 0) {
            prefetch_tensormap(&map_a);
            prefetch_tensormap(&map_b);
            int issued = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                int m, n;
                tm.at(t, m, n);
                for (int k = 0; k < ksteps; ++k, ++issued) {
                    const int s = issued % T::STAGES;
                    if (issued >= T::STAGES && !mbar_wait_bounded(&empty[s], uint32_t(issued / T::STAGES - 1) & 1u)) {
                        ok = false;
                        break;
                    }
                    uint8_t *st = stages + s * T::STAGE_BYTES;
                    mbar_arrive_expect_tx(&full[s], T::STAGE_BYTES);
                    tma_load_2d(st, &map_a, &full[s], k * BK, m * BM);
                    tma_load_2d(st + BM * BK * 2, &map_b, &full[s], k * BK, n * BN);
                }
            }
            if (!ok) {
                atomicOr(status, 1u);
                for (int i = max(0, issued - T::STAGES); i < issued; ++i)
                    mbar_wait_bounded(&full[i % T::STAGES], uint32_t(i / T::STAGES) & 1u);
            }
        }
    } else if (warp == 9) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_f16(BM, BN);
            int used = 0, filled = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                for (int c = 0; c < chunks && ok; ++c, ++filled) {
                    const int b = filled & 1;
                    if (filled >= 2 && !mbar_wait_bounded(&acc_empty[b], uint32_t(filled / 2 - 1) & 1u)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int k1 = min(ksteps, (c + 1) * kChunkSteps);
                    for (int k = c * kChunkSteps; k < k1; ++k, ++used) {
                        const int s = used % T::STAGES;
                        if (!mbar_wait_bounded(&full[s], uint32_t(used / T::STAGES) & 1u)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t st = smem_addr(stages + s * T::STAGE_BYTES);
                        const uint64_t da = smem_desc_sw128(st), db = smem_desc_sw128(st + BM * BK * 2);
#pragma unroll
                        for (int j = 0; j < BK / 16; ++j)      // 32 bytes of k a step within the swizzled row
                            tc_mma_f16(tmem + b * BN, da + 2 * j, db + 2 * j, idesc, k > c * kChunkSteps || j > 0);
                        tc_commit(&empty[s]);
                    }
                    if (ok) tc_commit(&acc_full[b]);
                }
            }
            if (!ok) {
                atomicOr(status, 1u);
                tc_commit(&drained);
                mbar_wait_bounded(&drained, 0u);
            }
        }
    } else {
        const int half = warp >> 2;                            // columns half * COLS .. of the tile
        const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
        float4 *block = reinterpret_cast<float4 *>(stages + T::STAGES * T::STAGE_BYTES + warp * T::WARP_STAGE);
        int drains = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            int tile_m, tile_n;
            tm.at(t, tile_m, tile_n);
            const int64_t row0 = int64_t(tile_m) * BM + 32 * (warp & 3), col0 = int64_t(tile_n) * BN + half * T::COLS;
            const float sa = row0 + lane < p.M ? __ldg(p.sa + row0 + lane) : 0.0f;
            int acc[T::COLS];
#pragma unroll
            for (int i = 0; i < T::COLS; ++i) acc[i] = 0;
            for (int c = 0; c < chunks; ++c, ++drains) {
                const int b = drains & 1;
                if (!mbar_wait_bounded(&acc_full[b], uint32_t(drains / 2) & 1u)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < T::COLS / 32; ++j) {
                    uint32_t v[32];
                    tmem_load32(tmem + lanes + b * BN + half * T::COLS + 32 * j, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) acc[32 * j + i] += __float2int_rn(__uint_as_float(v[i]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[b]);
            }
            if (!ok) {
                if (lane == 0) atomicOr(status, 1u);
                break;
            }
            // 32 columns at a time through the warp's block (16-byte chunk c of
            // row r in slot c ^ (r & 7)): a lane writes its row, then eight
            // lanes read a row's 128 bytes, so the stores are whole lines
#pragma unroll
            for (int j = 0; j < T::COLS / 32; ++j) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int *a = acc + 32 * j + 4 * c;
                    block[lane * 8 + (c ^ (lane & 7))] =
                        make_float4(__fmul_rn(__int2float_rn(a[0]), sa), __fmul_rn(__int2float_rn(a[1]), sa),
                                    __fmul_rn(__int2float_rn(a[2]), sa), __fmul_rn(__int2float_rn(a[3]), sa));
                }
                __syncwarp();
                constexpr int W = TY == REPOPS_TYPE_F32 ? 4 : 8;      // columns a lane stores at once
                constexpr int PER_ROW = 32 / W, ROWS = 32 / PER_ROW;
                const int cl = (lane % PER_ROW) * W;
                const int64_t col = col0 + 32 * j + cl;
                float sb[W], bi[W];
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    sb[i] = col + i < p.N ? __ldg(p.sb + col + i) : 0.0f;
                    bi[i] = p.bias && col + i < p.N ? __ldg(p.bias + col + i) : 0.0f;
                }
#pragma unroll
                for (int r0 = 0; r0 < 32; r0 += ROWS) {
                    const int r = r0 + lane / PER_ROW;
                    float v[W];
#pragma unroll
                    for (int i = 0; i < W / 4; ++i) {
                        const float4 f = block[r * 8 + ((cl / 4 + i) ^ (r & 7))];
                        v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
                    }
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        v[i] = __fmul_rn(v[i], sb[i]);
                        if (p.bias) v[i] = __fadd_rn(v[i], bi[i]);
                    }
                    const int64_t row = row0 + r;
                    if (row >= p.M) continue;
                    const int64_t at = row * p.ldc + col;
                    if (c_vec && col + W <= p.N) {
                        if constexpr (TY == REPOPS_TYPE_F32) {
                            *reinterpret_cast<float4 *>(static_cast<float *>(p.C) + at) = make_float4(v[0], v[1], v[2], v[3]);
                        } else {
                            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.C) + at) =
                                make_uint4(pack_c<TY>(v[0], v[1]), pack_c<TY>(v[2], v[3]), pack_c<TY>(v[4], v[5]),
                                           pack_c<TY>(v[6], v[7]));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < W; ++i)
                            if (col + i < p.N) store_c<TY>(p.C, at + i, v[i]);
                    }
                }
                __syncwarp();
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_free(tmem, T::TMEM_COLS);
}

// ------------------------------------------------------------------- host ----

enum I8Config { CFG_AUTO = -1, CFG_ROWS = 0, CFG_TILE256 = 1, CFG_TILE128 = 2, CFG_TILE64 = 3, CFG_COUNT = 4 };

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int sm_count() {
    DeviceInfo di;
    return current_device_info(&di) == REPOPS_OK ? di.sms : 152;
}

int64_t padded_k(int64_t K) { return ceil_div(K, BK) * BK; }

uint64_t tile_workspace(int64_t M, int64_t N, int64_t K) { return uint64_t(M + N) * uint64_t(padded_k(K)) * 2u; }

int auto_config(int64_t M, int64_t N, int64_t K) {
    if (M <= 64 || K == 0) return CFG_ROWS;
    return N > 128 ? CFG_TILE256 : N > 64 ? CFG_TILE128 : CFG_TILE64;
}

bool operand_vec(const int8_t *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 16 == 0; }

template <int TY, int MT, int NT>
int launch_rows_nt(const I8Args &a, cudaStream_t s) {
    const dim3 grid(unsigned(ceil_div(a.N, 16 * MT)), unsigned(ceil_div(a.M, 8 * NT)));
    if (operand_vec(a.A, a.lda) && operand_vec(a.B, a.ldb)) gemm_i8_rows_kernel<TY, MT, NT, true><<<grid, 256, 0, s>>>(a);
    else gemm_i8_rows_kernel<TY, MT, NT, false><<<grid, 256, 0, s>>>(a);
    return check_launch();
}

template <int TY>
int launch_rows(const I8Args &a, cudaStream_t s) {
    if (a.M <= 8) return launch_rows_nt<TY, 1, 1>(a, s);
    if (a.M <= 16) return launch_rows_nt<TY, 1, 2>(a, s);
    if (a.M <= 32) return launch_rows_nt<TY, 1, 4>(a, s);
    return launch_rows_nt<TY, 1, 8>(a, s);
}

bool make_map(CUtensorMap *map, const __half *base, int64_t Kp, int64_t rows, int box_rows) {
    gemm::EncodeTiledFn enc = gemm::tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {cuuint64_t(Kp), cuuint64_t(rows)}, strides[1] = {cuuint64_t(Kp) * 2u};
    const cuuint32_t box[2] = {cuuint32_t(BK), cuuint32_t(box_rows)}, estr[2] = {1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<__half *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int TY, int BN>
int launch_tile(const I8Args &a, __half *ws, cudaStream_t s) {
    using T = TileCfg<BN>;
    const int64_t Kp = padded_k(a.K);
    const int64_t items = (a.M + a.N) * (Kp / 16);
    const unsigned wgrid = unsigned(std::min<int64_t>(ceil_div(items, 256), int64_t(sm_count()) * 32));
    if (operand_vec(a.A, a.lda) && operand_vec(a.B, a.ldb)) widen_kernel<true><<<wgrid, 256, 0, s>>>(a, Kp, ws);
    else widen_kernel<false><<<wgrid, 256, 0, s>>>(a, Kp, ws);
    int rc = check_launch();
    if (rc != REPOPS_OK) return rc;
    CUtensorMap ma, mb;
    if (!make_map(&ma, ws, Kp, a.M, BM) || !make_map(&mb, ws + a.M * Kp, Kp, a.N, BN)) return REPOPS_ERR_UNSUPPORTED;
    unsigned *status = nullptr;
    if ((rc = status_word_address(&status)) != REPOPS_OK) return rc;
    auto kern = gemm_i8_tile_kernel<TY, BN>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
    if (e != cudaSuccess) return set_cuda_error(e);
    const TileMap tm{int(ceil_div(a.M, BM)), int(ceil_div(a.N, BN)), 16};
    const int64_t tiles = int64_t(tm.tiles_m) * tm.tiles_n;
    const unsigned csize = TY == REPOPS_TYPE_F32 ? 4u : 2u;
    const int c_vec = reinterpret_cast<uintptr_t>(a.C) % 16 == 0 && uint64_t(a.ldc) * csize % 16 == 0;
    kern<<<unsigned(std::min<int64_t>(tiles, sm_count())), kTileThreads, T::SMEM, s>>>(ma, mb, a, tm, int(Kp / BK),
                                                                                      c_vec, status);
    return check_launch();
}

template <int TY>
int run_i8(int cfg, const I8Args &a, void *ws, cudaStream_t s) {
    switch (cfg) {
        case CFG_ROWS: return launch_rows<TY>(a, s);
        case CFG_TILE256: return launch_tile<TY, 256>(a, static_cast<__half *>(ws), s);
        case CFG_TILE128: return launch_tile<TY, 128>(a, static_cast<__half *>(ws), s);
        default: return launch_tile<TY, 64>(a, static_cast<__half *>(ws), s);
    }
}

}  // namespace
}  // namespace repops

using namespace repops;

extern "C" int repops_gemm_i8_config_count(void) { return CFG_COUNT; }

extern "C" int repops_gemm_i8_auto_config(int64_t M, int64_t N, int64_t K) {
    return M < 0 || N < 0 || K < 0 ? REPOPS_ERR_INVALID_ARG : auto_config(M, N, K);
}

extern "C" uint64_t repops_gemm_i8_workspace_bytes(int config, int64_t M, int64_t N, int64_t K) {
    if (config < CFG_AUTO || config >= CFG_COUNT || M <= 0 || N <= 0 || K <= 0 || K > kMaxK ||
        M > (int64_t(1) << 40) || N > (int64_t(1) << 40))
        return 0;
    if (config == CFG_AUTO) config = auto_config(M, N, K);
    return config == CFG_ROWS ? 0 : tile_workspace(M, N, K);
}

extern "C" int repops_gemm_i8(int config, int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda,
                              const float *a_scale, const int8_t *B, int64_t ldb, const float *b_scale,
                              const float *bias, void *C, int typeC, int64_t ldc, void *ws, uint64_t ws_bytes,
                              cudaStream_t stream) {
    if (M < 0 || N < 0 || K < 0 || !known_storage(typeC) || config < CFG_AUTO || config >= CFG_COUNT)
        return REPOPS_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return REPOPS_OK;
    if (K > kMaxK) return REPOPS_ERR_UNSUPPORTED;
    if ((K > 0 && (!A || !B)) || !a_scale || !b_scale || !C) return REPOPS_ERR_INVALID_ARG;
    uint64_t ab, bb, cb;
    if (!span_bytes(M, K, lda, 1, &ab) || !span_bytes(N, K, ldb, 1, &bb) ||
        !span_bytes(M, N, ldc, storage_size(typeC), &cb))
        return REPOPS_ERR_INVALID_ARG;
    const uint64_t sab = uint64_t(M) * 4u, sbb = uint64_t(N) * 4u;
    if (ranges_overlap(C, cb, A, ab) || ranges_overlap(C, cb, B, bb) || ranges_overlap(C, cb, a_scale, sab) ||
        ranges_overlap(C, cb, b_scale, sbb) || (bias && ranges_overlap(C, cb, bias, sbb)))
        return REPOPS_ERR_ALIAS;
    if (config == CFG_AUTO) config = auto_config(M, N, K);
    if (K == 0) config = CFG_ROWS;
    // the grids' limits: tile indices are 32-bit, and a grid's y is at most 65535
    if (ceil_div(M, BM) * ceil_div(N, 16) > INT32_MAX / 2 || (config == CFG_ROWS && ceil_div(M, 64) > 65535))
        return REPOPS_ERR_UNSUPPORTED;
    const uint64_t need = repops_gemm_i8_workspace_bytes(config, M, N, K);
    void *own = nullptr;
    if (need > 0) {
        if (ws) {
            if (ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 16 != 0) return REPOPS_ERR_INVALID_ARG;
            if (ranges_overlap(ws, need, A, ab) || ranges_overlap(ws, need, B, bb) || ranges_overlap(ws, need, C, cb) ||
                ranges_overlap(ws, need, a_scale, sab) || ranges_overlap(ws, need, b_scale, sbb) ||
                (bias && ranges_overlap(ws, need, bias, sbb)))
                return REPOPS_ERR_ALIAS;
        } else {
            if (scratch_malloc(&own, size_t(need), stream) != cudaSuccess) {
                cudaGetLastError();
                return REPOPS_ERR_ALLOC;
            }
            ws = own;
        }
    }
    const I8Args a{M, N, K, A, B, lda, ldb, a_scale, b_scale, bias, C, ldc, A + ab, B + bb};
    int rc = typeC == REPOPS_TYPE_F32   ? run_i8<REPOPS_TYPE_F32>(config, a, ws, stream)
             : typeC == REPOPS_TYPE_F16 ? run_i8<REPOPS_TYPE_F16>(config, a, ws, stream)
                                        : run_i8<REPOPS_TYPE_BF16>(config, a, ws, stream);
    if (own) {
        const cudaError_t e = cudaFreeAsync(own, stream);
        if (rc == REPOPS_OK && e != cudaSuccess) rc = set_cuda_error(e);
    }
    return rc;
}
