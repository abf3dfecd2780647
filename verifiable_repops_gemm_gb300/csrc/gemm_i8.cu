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
// add their sums in shared memory.  The instruction's rate here is 130 TOPS
// (measured), enough for 8 tokens at the memory's rate; widening to binary16
// in registers for the faster-looking m16n8k16.f16 took 31 us where this takes
// 12 (16384 channels, 2048 k, 13 tokens).
//
// More rows: tcgen05 on binary16 (8 bits fit its 11) with binary32 accumulators
// in tensor memory.  Every product and every partial sum of up to 1024 of them is
// a whole number of at most 2^24, so binary32 accumulation is exact whatever its
// order; after each 1024 of k the accumulators are added to 32-bit integers in
// registers while the tensor core fills the other half of the accumulators'
// tensor memory.  (A conversion to integer takes 8 cycles a warp: 1000 cycles for
// a drain, against 4500 of products.)
//
// B streams through once as bytes and is widened on its way into tensor memory,
// where it is the product's first operand (128 channels x k): its binary16 form
// never passes through shared memory or DRAM.  (Widening both operands to scratch
// first reads and writes 5 bytes for each of B's: with that, 8192 x 8192 took 64
// us at 128 tokens and 214 at 2048, where this takes 22 and 180.)  The tokens are
// widened to scratch before and loaded by TMA.  Where there are fewer tiles than
// SMs a cluster shares a tile's k: each CTA leaves its 32-bit sums in shared
// memory, and after the cluster's barrier each adds and stores its share of the
// tokens.  (Adding parts by atomics in scratch took 23 us for 8192 x 8192, 64
// tokens; this takes 19.)  Bound: at 64 tokens by what is not the products, 7 us
// of launches, the tokens' widening, first loads and last stores, then by a step
// of the products (0.33 us for 128 of k, 128 channels and 64 tokens; B at 5 TB/s);
// at 2048 by the tensor cores (2048 x 16384 x 2048: 92 us, tensor pipe 71% active,
// 224 steps of 128 x 128 x 128 at 0.37 us).
//
// Thousands of rows: widening each channel once for every 128 tokens costs more
// than widening it once to scratch, above all in power.  Pairs of CTAs
// (cta_group::2, each reads half of B from its shared memory) multiply tiles of
// 256 x 256 from widened copies.  8192 x 8192 x 8192 takes 670 us: 59 to widen
// (6.8 TB/s), then 1.8 PFLOP/s, bound by the tensor cores at the clock the power
// limit leaves; the kernel above takes 690 (740 against 700 where L2 is cold).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gemm_common.h"
#include "internal.cuh"
#include "rows8.cuh"
#include "tcgen05.cuh"

namespace repops {
namespace {

constexpr int64_t kMaxK = 131071;

struct I8Args : DbgAccess {
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
__device__ __forceinline__ uint4 load_k16(const DbgAccess &d, const int8_t *__restrict__ row, int64_t k, int64_t n,
                                          const int8_t *base, const int8_t *end) {
    const int8_t *p = row + k;
    if (k + 16 <= n) {
        if constexpr (VEC) {
            return load_const(d, reinterpret_cast<const uint4 *>(p));
        } else {
            const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(p) & 3u);
            const int8_t *q = p - off;
            if (q >= base && q + (off ? 20 : 16) <= end) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(q);
                const uint32_t w0 = load_const(d, w), w1 = load_const(d, w + 1), w2 = load_const(d, w + 2),
                               w3 = load_const(d, w + 3), w4 = off ? load_const(d, w + 4) : 0u;
                const uint32_t s = 8 * off;
                return make_uint4(__funnelshift_r(w0, w1, s), __funnelshift_r(w1, w2, s), __funnelshift_r(w2, w3, s),
                                  __funnelshift_r(w3, w4, s));
            }
        }
    }
    uint32_t r[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (k + i < n) r[i >> 2] |= uint32_t(uint8_t(load_global(d, p + i))) << (8 * (i & 3));
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// 16 bytes that all lie within a row, without a branch: a guard around a load
// makes the loads of a loop wait for one another.  Where the address is not
// aligned, every word read holds at least one of the bytes asked for.
template <bool VEC>
__device__ __forceinline__ uint4 load_full16(const DbgAccess &d, const int8_t *__restrict__ p) {
    if constexpr (VEC) return load_const(d, reinterpret_cast<const uint4 *>(p));
    const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(p) & 3u), s = 8 * off;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(p - off);
    const uint32_t w0 = load_const(d, w), w1 = load_const(d, w + 1), w2 = load_const(d, w + 2), w3 = load_const(d, w + 3),
                   w4 = load_const(d, w + (off ? 4 : 3));
    return make_uint4(__funnelshift_r(w0, w1, s), __funnelshift_r(w1, w2, s), __funnelshift_r(w2, w3, s),
                      __funnelshift_r(w3, w4, s));
}
// ---------------------------------------------------------------- epilogue ----

template <int TY>
__device__ __forceinline__ void store_c(void *C, int64_t i, float v) {
    if constexpr (TY == REPOPS_TYPE_F32) static_cast<float *>(C)[i] = v;
    else if constexpr (TY == REPOPS_TYPE_F16) static_cast<__half *>(C)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(C)[i] = __float2bfloat16_rn(v);
}

// Element i of C, in global memory.
template <int TY>
__device__ __forceinline__ void store_c(const DbgAccess &d, void *C, int64_t i, float v) {
    constexpr uint32_t size = TY == REPOPS_TYPE_F32 ? 4u : 2u;
    if (REPOPS_DBG_WRITE(d, static_cast<const uint8_t *>(C) + i * int64_t(size), size)) store_c<TY>(C, i, v);
}

template <int TY>
__device__ __forceinline__ uint32_t pack_c(float lo, float hi) {
    uint16_t h[2];
    store_c<TY>(h, 0, lo);
    store_c<TY>(h, 1, hi);
    return h[0] | (uint32_t(h[1]) << 16);
}

__device__ __forceinline__ float scale_bias(const I8Args &p, float v, int64_t j) {
    v = __fmul_rn(v, load_const(p, p.sb + j));
    return p.bias ? __fadd_rn(v, load_const(p, p.bias + j)) : v;
}

// ---------------------------------------------------------------- few rows ----

// Whole numbers as binary16: with the sign bit flipped a byte is q + 128, the
// low mantissa bits of 1024 + (q + 128); subtracting 1152 is exact.
__device__ __forceinline__ uint32_t widen2(uint32_t w, uint32_t selector) {
    const uint32_t h = __byte_perm(w, 0x64646464u, selector);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&h), __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One or two (NT) tokens: a warp takes R channels, its lanes 512 consecutive bytes
// of each at once, and multiplies by dp4a: the tensor instruction's rate would
// be spent on columns that are not there (at 8192 x 8192 its eight take 8 of the
// 10 us that reading B takes).
template <int TY, int R, int NT, bool VEC>
__global__ void __launch_bounds__(256) gemm_i8_dot_kernel(I8Args p) {
    const int lane = threadIdx.x & 31;
    const int64_t j0 = (blockIdx.x * int64_t(8) + (threadIdx.x >> 5)) * R;
    if (j0 >= p.N) return;
    int acc[R][NT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < NT; ++m) acc[r][m] = 0;
    // a channel or token past the end repeats the last one, and is not stored
    const int8_t *rw[R], *rx[NT];
#pragma unroll
    for (int r = 0; r < R; ++r) rw[r] = p.B + min(j0 + r, p.N - 1) * p.ldb;
#pragma unroll
    for (int m = 0; m < NT; ++m) rx[m] = p.A + min(int64_t(m), p.M - 1) * p.lda;
    auto multiply = [&](const uint4 (&w)[R], const uint4 (&x)[NT]) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int m = 0; m < NT; ++m) {
                acc[r][m] = __dp4a(int(w[r].x), int(x[m].x), acc[r][m]);
                acc[r][m] = __dp4a(int(w[r].y), int(x[m].y), acc[r][m]);
                acc[r][m] = __dp4a(int(w[r].z), int(x[m].z), acc[r][m]);
                acc[r][m] = __dp4a(int(w[r].w), int(x[m].w), acc[r][m]);
            }
    };
    const int K = int(p.K);
    int k = 16 * lane;
#pragma unroll 8 / R
    for (; k + 16 <= K; k += 512) {
        uint4 w[R], x[NT];
#pragma unroll
        for (int r = 0; r < R; ++r) w[r] = load_full16<VEC>(p, rw[r] + k);
#pragma unroll
        for (int m = 0; m < NT; ++m) x[m] = load_full16<VEC>(p, rx[m] + k);
        multiply(w, x);
    }
    if (k < K) {
        uint4 w[R], x[NT];
#pragma unroll
        for (int r = 0; r < R; ++r) w[r] = load_k16<VEC>(p, rw[r], k, K, p.B, p.b_end);
#pragma unroll
        for (int m = 0; m < NT; ++m) x[m] = load_k16<VEC>(p, rx[m], k, K, p.A, p.a_end);
        multiply(w, x);
    }
    int mine = 0;                      // lane r * NT + m keeps channel r, token m
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < NT; ++m) {
            const int v = __reduce_add_sync(0xffffffffu, acc[r][m]);
            if (lane == r * NT + m) mine = v;
        }
    const int64_t j = j0 + lane / NT, m = lane % NT;
    if (lane < R * NT && j < p.N && m < p.M) {
        const float v = __fmul_rn(__int2float_rn(mine), load_const(p, p.sa + m));
        store_c<TY>(p, p.C, m * p.ldc + j, scale_bias(p, v, j));
    }
}

// 16 channels x 8 * NT tokens a CTA of 8 warps; warp w takes the 64-k steps w,
// w + 8, ...  (Two tiles of channels a warp were slower at every size but one.)  The
// instruction's latency is long: a step's two go to accumulators of their own (2048
// channels of 8192, 8 tokens: 12.2 -> 8.7 us), and with more than 8 tokens a step's
// loads in flight are enough (two or four took a warp's place on the SM: 16384 x
// 2048, 32 tokens 19.7, with two 23).
template <int TY, int NT, bool VEC>
__global__ void __launch_bounds__(256) gemm_i8_rows_kernel(I8Args p) {
    constexpr int CH = 16, TK = 8 * NT, PITCH = CH + 4;         // 2 * PITCH = 8 (mod 32): the adds hit 32 banks
    constexpr int UNROLL = NT == 1 ? 4 : 1;           // k-steps whose loads are in flight
    __shared__ int sum[TK][PITCH];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int64_t n0 = int64_t(blockIdx.x) * CH, m0 = int64_t(blockIdx.y) * TK;
    for (int i = threadIdx.x; i < TK * PITCH; i += 256) (&sum[0][0])[i] = 0;
    int d[NT][4], d2[NT][4];
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[u][i] = d2[u][i] = 0;
    // a channel or token past the end repeats the last one, and is not stored
    const int8_t *rw[2], *rx[NT];
#pragma unroll
    for (int h = 0; h < 2; ++h) rw[h] = p.B + min(n0 + 8 * h + g, p.N - 1) * p.ldb;
#pragma unroll
    for (int u = 0; u < NT; ++u) rx[u] = p.A + min(m0 + 8 * u + g, p.M - 1) * p.lda;
    const int full = int(p.K / 64);
    auto multiply = [&](const uint4 (&w)[2], const uint4 (&x)[NT]) {
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            mma_s8(d[u], w[0].x, w[1].x, w[0].y, w[1].y, x[u].x, x[u].y);
            mma_s8(d2[u], w[0].z, w[1].z, w[0].w, w[1].w, x[u].z, x[u].w);
        }
    };
    const int ahead = full - 8 * (UNROLL - 1);
    int s = warp;
    for (; s < ahead; s += 8 * UNROLL) {
        uint4 w[UNROLL][2], x[UNROLL][NT];
#pragma unroll
        for (int e = 0; e < UNROLL; ++e) {
            const int k = (s + 8 * e) * 64 + 16 * q;
#pragma unroll
            for (int h = 0; h < 2; ++h) w[e][h] = load_full16<VEC>(p, rw[h] + k);
#pragma unroll
            for (int u = 0; u < NT; ++u) x[e][u] = load_full16<VEC>(p, rx[u] + k);
        }
#pragma unroll
        for (int e = 0; e < UNROLL; ++e) multiply(w[e], x[e]);
    }
    for (; s < full; s += 8) {
        const int k = s * 64 + 16 * q;
        uint4 w[2], x[NT];
#pragma unroll
        for (int h = 0; h < 2; ++h) w[h] = load_full16<VEC>(p, rw[h] + k);
#pragma unroll
        for (int u = 0; u < NT; ++u) x[u] = load_full16<VEC>(p, rx[u] + k);
        multiply(w, x);
    }
    if (s == full && p.K % 64) {                               // the last step, in part behind K
        const int64_t k = int64_t(s) * 64 + 16 * q;
        uint4 w[2], x[NT];
#pragma unroll
        for (int h = 0; h < 2; ++h) w[h] = load_k16<VEC>(p, rw[h], k, p.K, p.B, p.b_end);
#pragma unroll
        for (int u = 0; u < NT; ++u) x[u] = load_k16<VEC>(p, rx[u], k, p.K, p.A, p.a_end);
        multiply(w, x);
    }
    __syncthreads();
    // lane: channels g and g + 8, tokens 2q and 2q + 1 of each tile
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            atomicAdd(&sum[8 * u + 2 * q + (i & 1)][8 * (i >> 1) + g], d[u][i] + d2[u][i]);
    __syncthreads();
    for (int i = threadIdx.x; i < TK * CH; i += 256) {
        const int64_t m = m0 + i / CH, n = n0 + i % CH;
        if (m >= p.M || n >= p.N) continue;
        const float v = __fmul_rn(__int2float_rn(sum[i / CH][i % CH]), load_const(p, p.sa + m));
        store_c<TY>(p, p.C, m * p.ldc + n, scale_bias(p, v, n));
    }
}

// --------------------------------------------------------------- more rows ----

constexpr int BM = 128;                   // channels of a tile
constexpr int kStreamK = 128;             // k of a step: a 128-byte row of B
constexpr int kStreamChunk = 1024 / kStreamK;        // steps between two drains: the most that stays exact
constexpr int kStreamThreads = 608;       // 8 epilogue warps, 8 widening warps, a TMA warp each for B and tokens, an MMA warp

// Bytes k .. k+7 of a row (zeros from `n` on), as load_k16 loads sixteen.
template <bool VEC>
__device__ __forceinline__ uint2 load_k8(const DbgAccess &d, const int8_t *__restrict__ row, int64_t k, int64_t n,
                                         const int8_t *base, const int8_t *end) {
    const int8_t *p = row + k;
    if (k + 8 <= n) {
        if constexpr (VEC) {
            return load_const(d, reinterpret_cast<const uint2 *>(p));
        } else {
            const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(p) & 3u);
            const int8_t *q = p - off;
            if (q >= base && q + (off ? 12 : 8) <= end) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(q);
                const uint32_t w0 = load_const(d, w), w1 = load_const(d, w + 1), w2 = off ? load_const(d, w + 2) : 0u;
                return make_uint2(__funnelshift_r(w0, w1, 8 * off), __funnelshift_r(w1, w2, 8 * off));
            }
        }
    }
    uint32_t r[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < n) r[i >> 2] |= uint32_t(uint8_t(load_global(d, p + i))) << (8 * (i & 3));
    return make_uint2(r[0], r[1]);
}

struct TileMap {
    int tiles_m, tiles_n, band;           // m: token tiles, walked `band` at a time for L2 reuse; n: channel tiles
    __device__ __forceinline__ void at(int t, int &m, int &n) const {
        const int per = band * tiles_n, b = t / per, first = b * band, rows = min(band, tiles_m - first);
        const int r = t - b * per;
        n = r / rows;
        m = first + r - n * rows;
    }
};

// BT tokens a tile.  Three rings: B's bytes (freed once widened), the tokens in
// shared memory and the widened channels in tensor memory (both freed by the
// products).  Tensor memory: two accumulators of BT columns, then 64 columns for
// each stage's widened channels.
template <int BT>
struct StreamCfg {
    static constexpr int W_BYTES = BM * kStreamK, BOX_BYTES = BT * 128, T_BYTES = 2 * BOX_BYTES;
    static constexpr int T_STAGES = 4;
    static constexpr int W_STAGES = (229376 - T_STAGES * T_BYTES) / W_BYTES;     // 10 or 6
    static constexpr int SMEM = 1024 + W_STAGES * W_BYTES + T_STAGES * T_BYTES;
    static constexpr int A_COL = 2 * BT;
    static constexpr int COLS = BT / 2;                          // an epilogue warp's tokens
    static_assert(A_COL + T_STAGES * kStreamK / 2 <= 512 && W_STAGES % 2 == 0 && T_STAGES % 2 == 0);
};

// `parts` CTAs share a tile (its cluster), CTA r the k-steps [first(r), first(r + 1)).
struct StreamMap {
    TileMap order;
    int tiles, ksteps, parts;
    int copies, rows;                  // of the widened tokens, and a copy's rows
    __device__ __forceinline__ int first(int r) const { return int(int64_t(ksteps) * r / parts); }
};

// Item `it` of rows of `per` items each: its row, and its place there in `c`.
__device__ __forceinline__ int64_t item_row(int64_t it, uint32_t per, bool small, uint32_t &c) {
    const int64_t r = small ? int64_t(uint32_t(it) / per) : it / per;
    c = uint32_t(it - r * per);
    return r;
}

// Widens the tokens (rows of Kp, `copies` times) and copies B to rows of Kp where
// COPY.  An item is 8 values (a warp's store then covers 512 consecutive bytes), or
// 16 bytes of B; two items a thread are in flight.
template <bool VEC, bool COPY>
__global__ void __launch_bounds__(256)
stream_prepare_kernel(I8Args p, int64_t Kp, int copies, __half *__restrict__ tokens, int8_t *__restrict__ copy) {
    grid_release();
    const int64_t i0 = blockIdx.x * int64_t(512) + threadIdx.x, stride = int64_t(gridDim.x) * 512;
    const uint32_t per = uint32_t(Kp / 8);
    const int64_t items = p.M * per;
    const bool small = items <= UINT32_MAX;
    for (int64_t i = i0; i < items; i += stride) {
        uint2 w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t c;                                        // past the end: the last one again
            const int64_t r = item_row(min(i + 256 * j, items - 1), per, small, c);
            w[j] = load_k8<VEC>(p, p.A + r * p.lda, int64_t(c) * 8, p.K, p.A, p.a_end);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (i + 256 * j >= items) continue;
            const uint32_t a = w[j].x ^ 0x80808080u, b = w[j].y ^ 0x80808080u;
            const uint4 h = make_uint4(widen2(a, 0x4140u), widen2(a, 0x4342u), widen2(b, 0x4140u), widen2(b, 0x4342u));
            for (int64_t c = 0; c < copies; ++c) store_global(p, reinterpret_cast<uint4 *>(tokens + (i + 256 * j + c * items) * 8), h);
        }
    }
    if constexpr (COPY) {
        const uint32_t per16 = uint32_t(Kp / 16);
        const int64_t chunks = p.N * per16;
        const bool few = chunks <= UINT32_MAX;
        for (int64_t i = i0; i < chunks; i += stride) {
            uint4 w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t c;
                const int64_t r = item_row(min(i + 256 * j, chunks - 1), per16, few, c);
                w[j] = load_k16<false>(p, p.B + r * p.ldb, int64_t(c) * 16, p.K, p.B, p.b_end);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (i + 256 * j < chunks) store_global(p, reinterpret_cast<uint4 *>(copy) + i + 256 * j, w[j]);
        }
    }
}

template <int TY, int BT>
__global__ void __launch_bounds__(kStreamThreads, 1)
gemm_i8_stream_kernel(const __grid_constant__ CUtensorMap map_t, const __grid_constant__ CUtensorMap map_w, I8Args p,
                      StreamMap sm, int b_in_place, int c_vec, unsigned *status) {
    using T = StreamCfg<BT>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t w_full[T::W_STAGES], w_empty[T::W_STAGES];
    __shared__ uint64_t ready[T::T_STAGES], used[T::T_STAGES], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_slot;
    if (!REPOPS_DBG_SMEM_OK(T::SMEM, status)) return;
    uint8_t *w_ring = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u), *t_ring = w_ring + T::W_STAGES * T::W_BYTES;
    // from a shuffle the compiler knows that a warp's role is uniform: a product
    // is then issued in its own time, not in the 111 cycles that a branch it must
    // assume divergent costs
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = sm.parts == 1 ? 0 : int(cluster_rank());
    const int tile0 = int(blockIdx.x) / sm.parts, stride = int(gridDim.x) / sm.parts;
    const int k0 = sm.first(rank), steps = sm.first(rank + 1) - k0;     // of every tile
    if (threadIdx.x == 0) {
        for (int s = 0; s < T::W_STAGES; ++s) {
            mbar_init(&w_full[s], 1);
            mbar_init(&w_empty[s], 4);
        }
        for (int s = 0; s < T::T_STAGES; ++s) {
            mbar_init(&ready[s], 5);                           // the tokens' copy and four widening warps
            mbar_init(&used[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);
        }
        mbar_init(&drained, 1);
        fence_barrier_init();
    }
    if (warp == 18) tmem_alloc<1>(&tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);

    // Every wait gives up after its limit: the role that gave up sets the
    // status word, waits (again with a limit) for its own copies or products in
    // flight and leaves; the others run into their own limits.
    if (warp == 16 || warp == 17) {
        if (elect_one()) {
            const bool weights = warp == 16;
            const int stages = weights ? T::W_STAGES : T::T_STAGES;
            uint64_t *full = weights ? w_full : ready, *empty = weights ? w_empty : used;
            prefetch_tensormap(weights ? &map_w : &map_t);
            // B in place does not depend on the kernel before
            if (!weights || !b_in_place) grid_wait();
            int s = 0, issued = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int t = tile0; t < sm.tiles && ok; t += stride) {
                int ch, tok;
                sm.order.at(t, tok, ch);
                int k = k0 + ch % steps;                       // channels apart in k: not all on the same tokens
                for (int i = 0; i < steps; ++i, ++issued) {
                    if (!mbar_wait_bounded(&empty[s], phase)) {
                        ok = false;
                        break;
                    }
                    if (weights) {
                        mbar_arrive_expect_tx(&full[s], T::W_BYTES);
                        tma_load_2d(w_ring + s * T::W_BYTES, &map_w, &full[s], k * kStreamK, ch * BM);
                    } else {
                        mbar_arrive_expect_tx(&full[s], T::T_BYTES);
                        tma_load_3d(t_ring + s * T::T_BYTES, &map_t, &full[s], 0, tok * BT + int(blockIdx.x % sm.copies) * sm.rows, 2 * k);
                    }
                    if (++k == k0 + steps) k = k0;
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                atomicOr(status, 1u);
                for (int i = max(0, issued - stages); i < issued; ++i)
                    mbar_wait_bounded(&full[i % stages], uint32_t(i / stages) & 1u);
            }
        }
    } else if (warp == 18) {
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_f16(BM, BT);
            const uint32_t base = smem_addr(t_ring);
            int s = 0, b = 0;
            uint32_t phase = 0, acc_phase = 1;
            bool ok = true;
            for (int t = tile0; t < sm.tiles && ok; t += stride) {
                for (int c = 0; c < steps && ok; c += kStreamChunk) {
                    if (!mbar_wait_bounded(&acc_empty[b], acc_phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int n = min(kStreamChunk, steps - c);
                    for (int i = 0; i < n; ++i) {
                        if (!mbar_wait_bounded(&ready[s], phase)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t a = tmem + T::A_COL + s * (kStreamK / 2);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint64_t db = smem_desc_sw128(base + s * T::T_BYTES + h * T::BOX_BYTES);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                tc_mma_f16_tmem(tmem + b * BT, a + 32 * h + 8 * j, db + 2 * j, idesc,
                                                i > 0 || h > 0 || j > 0);
                        }
                        tc_commit<1>(&used[s]);
                        if (++s == T::T_STAGES) {
                            s = 0;
                            phase ^= 1u;
                        }
                    }
                    if (ok) tc_commit<1>(&acc_full[b]);
                    b ^= 1;
                    if (b == 0) acc_phase ^= 1u;
                }
            }
            if (!ok) {
                atomicOr(status, 1u);
                tc_commit<1>(&drained);
                mbar_wait_bounded(&drained, 0u);
            }
        }
    } else if (warp >= 8) {
        // four warps widen the even steps, four the odd: a lane its channel
        const int row = 32 * (warp & 3) + lane, n = steps * ((sm.tiles - tile0 + stride - 1) / stride);
        const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
        int sw = (warp - 8) >> 2, sa = sw;
        uint32_t w_phase = 0, a_phase = 1;
        for (int i = sw; i < n; i += 2) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&w_full[sw], w_phase) && mbar_wait_bounded(&used[sa], a_phase))) {
                if (lane == 0) atomicOr(status, 1u);
                break;
            }
            tc_fence_after();                                  // the products that read this stage's columns
            const uint8_t *st = w_ring + sw * T::W_BYTES + row * kStreamK;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(st + (((4 * h + c) ^ (row & 7)) << 4));
                    const uint32_t q[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[8 * c + 2 * e] = widen2(q[e], 0x4140u);
                        v[8 * c + 2 * e + 1] = widen2(q[e], 0x4342u);
                    }
                }
                tmem_store32(tmem + lanes + T::A_COL + sa * (kStreamK / 2) + 32 * h, v);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&w_empty[sw]);          // the warp has read its rows
            tmem_store_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ready[sa]);
            sw += 2;
            if (sw >= T::W_STAGES) {
                sw -= T::W_STAGES;
                w_phase ^= 1u;
            }
            sa += 2;
            if (sa >= T::T_STAGES) {
                sa -= T::T_STAGES;
                a_phase ^= 1u;
            }
        }
    } else {
        const int half = warp >> 2;                            // tokens half * COLS .. of the tile
        const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
        int b = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = tile0; t < sm.tiles; t += stride) {
            int ch, tok;
            sm.order.at(t, tok, ch);
            const int64_t n = int64_t(ch) * BM + 32 * (warp & 3) + lane, m0 = int64_t(tok) * BT + half * T::COLS;
            const int64_t nn = min(n, p.N - 1);                // past the end: not stored
            const float sb = load_const(p, p.sb + nn), bias = p.bias ? load_const(p, p.bias + nn) : 0.0f;
            float sa[T::COLS / 32];
#pragma unroll
            for (int i = 0; i < T::COLS / 32; ++i) sa[i] = load_const(p, p.sa + min(m0 + 32 * i + lane, p.M - 1));
            int acc[T::COLS];
#pragma unroll
            for (int i = 0; i < T::COLS; ++i) acc[i] = 0;
            for (int c = 0; c < steps; c += kStreamChunk) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&acc_full[b], phase));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < T::COLS; j += 16) {
                    uint32_t v[16];
                    tmem_load16(tmem + lanes + b * BT + half * T::COLS + j, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[j + i] += __float2int_rn(__uint_as_float(v[i]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[b]);
                b ^= 1;
                if (b == 0) phase ^= 1u;
            }
            if (!ok) {
                if (lane == 0) atomicOr(status, 1u);
                break;
            }
            if (sm.parts > 1) {
                // the only tile: every copy into the ring of B has been read
                int *sum = reinterpret_cast<int *>(w_ring) + half * T::COLS * BM + 32 * (warp & 3) + lane;
#pragma unroll
                for (int i = 0; i < T::COLS; ++i) sum[i * BM] = acc[i];
                break;
            }
            const int rows = n < p.N ? int(min(p.M - m0, int64_t(T::COLS))) : 0;
            using E = typename std::conditional<TY == REPOPS_TYPE_F32, float, uint16_t>::type;
            E *out = static_cast<E *>(p.C) + m0 * p.ldc + n;
            const bool add = p.bias != nullptr;
#pragma unroll
            for (int i = 0; i < T::COLS; ++i) {
                float v = __fmul_rn(__fmul_rn(__int2float_rn(acc[i]), __shfl_sync(0xffffffffu, sa[i / 32], i % 32)), sb);
                const float w = __fadd_rn(v, bias);
                v = add ? w : v;
                if (i < rows) store_c<TY>(p, out, 0, v);
                out += p.ldc;
            }
        }
    }
    if (sm.parts > 1) {
        // this CTA's tokens of the tile: rank, rank + parts, ...; a warp a token,
        // four channels a lane
        int ch, tok;
        sm.order.at(tile0, tok, ch);
        const int64_t n = int64_t(ch) * BM + 4 * lane, m0 = int64_t(tok) * BT;
        float sb[4], bias[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t nn = min(n + i, p.N - 1);
            sb[i] = load_const(p, p.sb + nn);
            bias[i] = p.bias ? load_const(p, p.bias + nn) : 0.0f;
        }
        __syncwarp();
        cluster_sync();
        for (int i = rank + sm.parts * warp; i < BT && m0 + i < p.M; i += sm.parts * (kStreamThreads / 32)) {
            const uint32_t at = uint32_t(i * BM + 4 * lane) * 4u;
            int4 v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < sm.parts) v[r] = load_cluster16(cluster_addr(w_ring, uint32_t(r)) + at);
            const float sa = load_const(p, p.sa + m0 + i);
            int4 a = v[0];
#pragma unroll
            for (int r = 1; r < 8; ++r)
                if (r < sm.parts) a = make_int4(a.x + v[r].x, a.y + v[r].y, a.z + v[r].z, a.w + v[r].w);
            float f[4] = {__int2float_rn(a.x), __int2float_rn(a.y), __int2float_rn(a.z), __int2float_rn(a.w)};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[j] = __fmul_rn(__fmul_rn(f[j], sa), sb[j]);
                if (p.bias) f[j] = __fadd_rn(f[j], bias[j]);
            }
            const int64_t o = (m0 + i) * p.ldc + n;
            if (c_vec && n + 4 <= p.N) {
                if constexpr (TY == REPOPS_TYPE_F32)
                    store_global(p, reinterpret_cast<float4 *>(static_cast<float *>(p.C) + o),
                                 make_float4(f[0], f[1], f[2], f[3]));
                else
                    store_global(p, reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.C) + o),
                                 make_uint2(pack_c<TY>(f[0], f[1]), pack_c<TY>(f[2], f[3])));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < p.N) store_c<TY>(p, p.C, o + j, f[j]);
            }
        }
        __syncwarp();
        cluster_sync();                                        // no CTA leaves while another reads its sums
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 18) tmem_free<1>(tmem, 512);
}

// ------------------------------------------------------------ thousands of rows ----

// With thousands of tokens the widening of B pays even through DRAM: a pair of CTAs
// multiplies a tile of 256 tokens x 256 channels from widened copies of both
// operands, and a stage's 64 KB feed twice the products that they feed above.
constexpr int BK = 64;                    // BK binary16 = one 128-byte swizzled row
constexpr int kPairChunk = 1024 / BK;     // k-steps between two drains
constexpr int kPairThreads = 320;         // 8 epilogue warps, a TMA warp, an MMA warp

struct PairCfg {
    static constexpr int BN = 256, B_ROWS = BN / 2;
    static constexpr int STAGE_BYTES = (BM + B_ROWS) * BK * 2;
    static constexpr int STAGES = 6;
    static constexpr int WARP_STAGE = 32 * 128;                  // an epilogue warp's block: 32 rows of 128 bytes
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + 8 * WARP_STAGE;
    static constexpr uint32_t TMEM_COLS = 2 * BN;
    static constexpr int COLS = BN / 2;                          // an epilogue warp's columns
};

// The rows of A, then those of B, as binary16 rows of Kp (a multiple of 64)
// values, zeros past K.  An item is 8 values, so that a warp's store covers 512
// consecutive bytes (16 values an item, stored as two halves of each 32-byte
// sector, took a third longer); two items a thread are in flight.
template <bool VEC>
__global__ void __launch_bounds__(256) widen_kernel(I8Args p, int64_t Kp, __half *__restrict__ out) {
    grid_release();
    const uint32_t per = uint32_t(Kp / 8);
    const int64_t items = (p.M + p.N) * per, stride = int64_t(gridDim.x) * 512;
    for (int64_t i0 = blockIdx.x * int64_t(512) + threadIdx.x; i0 < items; i0 += stride) {
        uint2 w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t it = min(i0 + 256 * j, items - 1);       // past the end: the last one again
            const int64_t r = items <= UINT32_MAX ? uint32_t(it) / per : it / per;
            const int64_t k = (it - r * per) * 8;
            w[j] = r < p.M ? load_k8<VEC>(p, p.A + r * p.lda, k, p.K, p.A, p.a_end)
                           : load_k8<VEC>(p, p.B + (r - p.M) * p.ldb, k, p.K, p.B, p.b_end);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (i0 + 256 * j >= items) continue;
            const uint32_t a = w[j].x ^ 0x80808080u, b = w[j].y ^ 0x80808080u;
            store_global(p, reinterpret_cast<uint4 *>(out + (i0 + 256 * j) * 8),
                         make_uint4(widen2(a, 0x4140u), widen2(a, 0x4342u), widen2(b, 0x4140u), widen2(b, 0x4342u)));
        }
    }
}

// C's tile: sums x scales, through the warp's block of shared memory.  Lane l
// holds the scales (and biases) of columns l, l + 32, ...  c_tma: C can be
// stored by TMA (a block of 32 rows x 128 bytes at a time, clipped at C's
// edges); else lanes store single values.
template <int TY, int COLS>
__device__ __forceinline__ void store_tile(const I8Args &p, const CUtensorMap *map_c, const int (&acc)[COLS], float sa,
                                           const float (&sb)[COLS / 32], const float (&bias)[COLS / 32], int64_t row0,
                                           int64_t col0, uint8_t *block, bool c_tma) {
    constexpr int W = TY == REPOPS_TYPE_F32 ? 32 : 64;         // columns of a block
    const int lane = threadIdx.x & 31;
    uint4 *chunk = reinterpret_cast<uint4 *>(block);           // 16-byte chunk c of row r in slot c ^ (r & 7)
#pragma unroll
    for (int j = 0; j < COLS; j += W) {
        if (col0 + j >= p.N) break;
        if (c_tma && lane == 0) tma_store_wait_read();         // the block's previous contents have left
        __syncwarp();
#pragma unroll
        for (int c = j; c < j + W; c += 8) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = __fmul_rn(__fmul_rn(__int2float_rn(acc[c + i]), sa),
                                 __shfl_sync(0xffffffffu, sb[c / 32], (c + i) % 32));
            if (p.bias) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = __fadd_rn(v[i], __shfl_sync(0xffffffffu, bias[c / 32], (c + i) % 32));
            }
            if constexpr (TY == REPOPS_TYPE_F32) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    chunk[lane * 8 + (((c - j) / 4 + h) ^ (lane & 7))] =
                        make_uint4(__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]),
                                   __float_as_uint(v[4 * h + 3]));
            } else {
                chunk[lane * 8 + (((c - j) / 8) ^ (lane & 7))] = make_uint4(
                    pack_c<TY>(v[0], v[1]), pack_c<TY>(v[2], v[3]), pack_c<TY>(v[4], v[5]), pack_c<TY>(v[6], v[7]));
            }
        }
        if (c_tma) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0 && row0 < p.M) tma_store_2d(map_c, block, int32_t(col0 + j), int32_t(row0));
        } else {
            __syncwarp();
            using E = typename std::conditional<TY == REPOPS_TYPE_F32, float, uint16_t>::type;
            constexpr int PER = 16 / int(sizeof(E));           // values of a chunk
            const E *e = reinterpret_cast<const E *>(block);
            const int rows = int(min(p.M - row0, int64_t(32)));
#pragma unroll
            for (int h = 0; h < W; h += 32) {
                const int c = h + lane;
                E *out = static_cast<E *>(p.C) + row0 * p.ldc + col0 + j + c;
                const bool mine = col0 + j + c < p.N;
#pragma unroll 8
                for (int r = 0; r < 32; ++r) {
                    const E v = e[(r * 8 + ((c / PER) ^ (r & 7))) * PER + c % PER];
                    if (mine && r < rows) store_global(p, out + r * p.ldc, v);
                }
            }
            __syncwarp();
        }
    }
}

template <int TY>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
gemm_i8_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                    const __grid_constant__ CUtensorMap map_c, I8Args p, TileMap tm, int ksteps, int c_tma,
                    unsigned *status) {
    using T = PairCfg;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[T::STAGES], empty[T::STAGES], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_slot;
    if (!REPOPS_DBG_SMEM_OK(T::SMEM, status)) return;
    uint8_t *stages = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int tiles = tm.tiles_m * tm.tiles_n, first = blockIdx.x / 2, stride = gridDim.x / 2;
    const int chunks = (ksteps + kPairChunk - 1) / kPairChunk;
    if (threadIdx.x == 0) {
        for (int s = 0; s < T::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 16);
        }
        mbar_init(&drained, 1);
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc<2>(&tmem_slot, T::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    grid_wait();                                               // the widened operands

    // Every wait gives up after its limit, as in the kernel above.
    if (warp == 8) {
        if (elect_one()) {
            prefetch_tensormap(&map_a);
            prefetch_tensormap(&map_b);
            int issued = 0, s = 0;
            uint32_t phase = 1;                                // the wait before the ring's first use passes
            bool ok = true;
            for (int t = first; t < tiles && ok; t += stride) {
                int m, n;
                tm.at(t, m, n);
                const int row_a = (m * 2 + int(rank)) * BM, row_b = n * T::BN + int(rank) * T::B_ROWS;
                for (int k = 0; k < ksteps; ++k, ++issued) {
                    if (!mbar_wait_bounded(&empty[s], phase)) {
                        ok = false;
                        break;
                    }
                    uint8_t *st = stages + s * T::STAGE_BYTES;
                    // a pair's four copies all signal the first CTA, whose
                    // barrier is armed for both CTAs' bytes; a copy of the other
                    // CTA that lands before that leaves the phase open, as the
                    // arming arrival is still missing
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * T::STAGE_BYTES);
                    const uint32_t bar = cluster_addr(&full[s], 0);
                    tma_load_2d_pair(st, &map_a, bar, k * BK, row_a);
                    tma_load_2d_pair(st + BM * BK * 2, &map_b, bar, k * BK, row_b);
                    if (++s == T::STAGES) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                atomicOr(status, 1u);
                if (rank == 0) {
                    for (int i = max(0, issued - T::STAGES); i < issued; ++i)
                        mbar_wait_bounded(&full[i % T::STAGES], uint32_t(i / T::STAGES) & 1u);
                } else {
                    // these copies signal the other CTA: give them the time of
                    // a copy a thousand times over
                    const uint64_t t0 = global_timer_ns();
                    while (global_timer_ns() - t0 < 2000000u) {}
                }
            }
        }
    } else if (warp == 9) {
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = idesc_f16(2 * BM, T::BN);
            const uint32_t base = smem_addr(stages);
            int s = 0, b = 0;
            uint32_t phase = 0, acc_phase = 1;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += stride) {
                for (int c = 0; c < chunks && ok; ++c) {
                    if (!mbar_wait_bounded(&acc_empty[b], acc_phase)) {
                        ok = false;
                        break;
                    }
                    asm volatile("fence.acq_rel.cluster;" ::: "memory");
                    tc_fence_after();
                    const int steps = min(kPairChunk, ksteps - c * kPairChunk);
                    for (int k = 0; k < steps; ++k) {
                        if (!mbar_wait_bounded(&full[s], phase)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t st = base + s * T::STAGE_BYTES;
                        const uint64_t da = smem_desc_sw128(st), db = smem_desc_sw128(st + BM * BK * 2);
#pragma unroll
                        for (int j = 0; j < BK / 16; ++j)      // 32 bytes of k a step within the swizzled row
                            tc_mma_f16_pair(tmem + b * T::BN, da + 2 * j, db + 2 * j, idesc, k > 0 || j > 0);
                        tc_commit<2>(&empty[s]);
                        if (++s == T::STAGES) {
                            s = 0;
                            phase ^= 1u;
                        }
                    }
                    if (ok) tc_commit<2>(&acc_full[b]);
                    b ^= 1;
                    if (b == 0) acc_phase ^= 1u;
                }
            }
            if (!ok) {
                atomicOr(status, 1u);
                tc_commit<2>(&drained);
                mbar_wait_bounded(&drained, 0u);
            }
        }
    } else {
        const int half = warp >> 2;                            // columns half * COLS .. of the tile
        const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
        uint8_t *block = stages + T::STAGES * T::STAGE_BYTES + warp * T::WARP_STAGE;
        int b = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += stride) {
            int tile_m, tile_n;
            tm.at(t, tile_m, tile_n);
            const int64_t row0 = (int64_t(tile_m) * 2 + rank) * BM + 32 * (warp & 3),
                          col0 = int64_t(tile_n) * T::BN + half * T::COLS;
            const float sa = load_const(p, p.sa + min(row0 + lane, p.M - 1));
            float sb[T::COLS / 32], bias[T::COLS / 32];
#pragma unroll
            for (int i = 0; i < T::COLS / 32; ++i) {
                const int64_t col = min(col0 + 32 * i + lane, p.N - 1);    // past the end: not stored
                sb[i] = load_const(p, p.sb + col);
                bias[i] = p.bias ? load_const(p, p.bias + col) : 0.0f;
            }
            int acc[T::COLS];
#pragma unroll
            for (int i = 0; i < T::COLS; ++i) acc[i] = 0;
            for (int c = 0; c < chunks; ++c) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&acc_full[b], phase));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < T::COLS; j += 16) {
                    uint32_t v[16];
                    tmem_load16(tmem + lanes + b * T::BN + half * T::COLS + j, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[j + i] += __float2int_rn(__uint_as_float(v[i]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(&acc_empty[b], 0));
                b ^= 1;
                if (b == 0) phase ^= 1u;
            }
            if (!ok) {
                if (lane == 0) atomicOr(status, 1u);
                break;
            }
            store_tile<TY, T::COLS>(p, &map_c, acc, sa, sb, bias, row0, col0, block, c_tma != 0);
        }
        if (c_tma && lane == 0) tma_store_wait();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();                   // no CTA leaves while the other may signal it
    tc_fence_after();
    if (warp == 9) tmem_free<2>(tmem, T::TMEM_COLS);
}

// ------------------------------------------------------------------- host ----

enum I8Config { CFG_AUTO = -1, CFG_ROWS, CFG_TILES, CFG_PAIR, CFG_COUNT };

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int sm_count() {
    DeviceInfo di;
    return current_device_info(&di) == REPOPS_OK ? di.sms : 152;
}

int64_t padded_k(int64_t K) { return ceil_div(K, BK) * BK; }

uint64_t pair_workspace(int64_t M, int64_t N, int64_t K) { return uint64_t(M + N) * uint64_t(padded_k(K)) * 2u; }

int64_t stream_k(int64_t K) { return ceil_div(K, kStreamK) * kStreamK; }

// Tokens a tile.
int stream_tokens(int64_t M) { return M <= 64 ? 64 : 128; }

// The largest cluster whose CTAs are all resident at once for every tile, and no
// more than one a k-step.  Clusters of one size that fit on the chip together:
// measured, and fixed so that a product's split does not depend on the device.
int stream_parts(int64_t tiles, int64_t ksteps) {
    constexpr int64_t fit[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
    int p = 1;
    for (int i = 2; i <= 8; ++i)
        if (tiles <= fit[i] && i <= ksteps) p = i;
    return p;
}

// Copies of the widened tokens.  Every CTA reads them all: where they are fewer
// than 128 KB they lie in too few slices of L2 (N 16384, K 2048: 12 us from 32
// tokens on, 16 with 8, and 12 with 8 in sixteen copies, a CTA reading one).
int stream_copies(int64_t M, int64_t K) {
    return int(std::clamp<int64_t>((int64_t(256) << 10) / (M * stream_k(K) * 2), 1, 16));
}

StreamMap stream_map(int64_t M, int64_t N, int64_t K) {
    StreamMap sm;
    // a band of 8 token tiles (2 bytes a value) by 19 of channels (1) in flight
    // on 152 SMs reads the fewest bytes
    sm.order = TileMap{int(ceil_div(M, stream_tokens(M))), int(ceil_div(N, BM)), 8};
    sm.ksteps = int(ceil_div(K, kStreamK));
    sm.tiles = sm.order.tiles_m * sm.order.tiles_n;
    sm.copies = stream_copies(M, K);
    sm.rows = int(M);
    sm.parts = stream_parts(sm.tiles, sm.ksteps);
    return sm;
}

// Scratch: the tokens in binary16; and a copy of B at a 16-byte pitch where TMA
// cannot read it in place.
uint64_t stream_workspace(int64_t M, int64_t K) {
    return uint64_t(M) * uint64_t(stream_copies(M, K)) * uint64_t(stream_k(K)) * 2u;
}
uint64_t stream_copy_bytes(int64_t N, int64_t K) { return uint64_t(N) * uint64_t(stream_k(K)); }

// The kernel whose estimated time is least, in us.
// Few rows: a fixed 3 and the memory's rate (5.9 TB/s here) or the integer tensor
// rate (115 TOPS in whole groups of 8 tokens), or a warp's k-steps one after
// another (0.45 each, longer with more tokens); 1.8 times that where K leaves rows
// off a 16-byte boundary.  Tiles: 7 (9 with 128 tokens a tile) of launches, fill and
// last store, a CTA's steps of 128 of k at 0.34 (0.38 with 128), the widening of
// many tokens and the copy of such rows of B.  Pairs: 8, the widening, and the
// waves of tiles x steps of 64 of k at 0.342.
// Measured either side, few rows and tiles: N = K = 2048: M 32 5.3, 7.9; M 64 9.6,
// 8.5.  N 16384, K 2048: M 16 11.9, 12.1; M 24 19.7, 12.1.  N = K = 8192: M 8 14.3,
// 18.2; M 16 24.3, 18.4.  N 2048, K 8192: M 8 8.7, 10.5; M 16 14.5, 10.7.  N 1023, K
// 3001: M 8 7.7, 9.0; M 16 10.2, 9.1.  Tiles and pairs: N = K = 8192: M 2048 179,
// 214; M 4096 352, 363; M 8192 690, 669.  N 16384, K 2048: M 2048 92, 100; M 8192
// 356, 350.  N 1023, K 3001: M 4097 35.5, 36.5.  One or two tokens have a kernel of
// their own.
int auto_config(int64_t M, int64_t N, int64_t K) {
    if (K == 0 || M <= 2) return CFG_ROWS;
    const double nk = double(N) * double(K), mk = double(M) * double(K), bt = stream_tokens(M);
    const double odd = K % 16 ? 1.0 : 0.0;
    const double rate = std::max(nk / 5.9e6, 2.0 * nk * double(ceil_div(M, 8) * 8) / 115e6) + 3.0;
    const double slower = M <= 8 ? 1.0 : M <= 16 ? 1.8 : M <= 32 ? 2.1 : 4.2 * double(ceil_div(M, 64));
    const double serial = 1.5 + 0.45 * double(ceil_div(K, 512)) * slower;
    const double few = std::max(rate, serial) * (1.0 + 0.8 * odd);
    const double tiles = double(ceil_div(N, BM)) * std::ceil(double(M) / bt);
    const double parts = stream_parts(int64_t(std::min(tiles, 1e6)), ceil_div(K, kStreamK));
    const double steps = std::ceil(tiles * parts / 152.0) * std::ceil(double(ceil_div(K, kStreamK)) / parts);
    const double many = (bt == 64 ? 7.2 + 0.34 * steps : 9.0 + 0.38 * steps) + std::max(0.0, 3.0 * mk / 5.5e6 - 3.0) +
                        odd * nk / 2.5e6;
    const double waves = std::ceil(double(ceil_div(M, 256)) * double(ceil_div(N, 256)) / 76.0);
    const double pairs = 8.0 + 3.0 * (nk + mk) / 5.5e6 + 0.342 * waves * double(ceil_div(K, BK)) + odd * (nk + mk) / 2.5e6;
    if (few <= many && few <= pairs) return CFG_ROWS;
    return many <= pairs ? CFG_TILES : CFG_PAIR;
}

// The kernel that a call runs, CFG_ROWS where there is nothing to multiply or
// the call is refused.
int run_config(int config, int64_t M, int64_t N, int64_t K) {
    if (config < CFG_AUTO || config >= CFG_COUNT || M <= 0 || N <= 0 || K <= 0 || K > kMaxK ||
        M > (int64_t(1) << 40) || N > (int64_t(1) << 40))
        return CFG_ROWS;
    return config == CFG_AUTO ? auto_config(M, N, K) : config;
}

bool operand_vec(const int8_t *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 16 == 0; }

// TMA reads B where it lies.
bool read_in_place(const int8_t *B, int64_t ldb) { return operand_vec(B, ldb) && ldb < (int64_t(1) << 39); }

template <int TY, int R, int NT>
int launch_dot(const I8Args &a, cudaStream_t s) {
    const unsigned grid = unsigned(ceil_div(a.N, 8 * R));
    if (operand_vec(a.A, a.lda) && operand_vec(a.B, a.ldb)) gemm_i8_dot_kernel<TY, R, NT, true><<<grid, 256, 0, s>>>(a);
    else gemm_i8_dot_kernel<TY, R, NT, false><<<grid, 256, 0, s>>>(a);
    return check_launch();
}

template <int TY, int R>
int launch_dot_r(const I8Args &a, cudaStream_t s) {
    return a.M == 1 ? launch_dot<TY, R, 1>(a, s) : launch_dot<TY, R, 2>(a, s);
}

// As many launches as a grid's 65535 token tiles make of M.
template <int TY, int NT>
int launch_rows_nt(I8Args a, cudaStream_t s) {
    constexpr int64_t most = int64_t(65535) * 8 * NT;
    const bool vec = operand_vec(a.A, a.lda) && operand_vec(a.B, a.ldb);
    for (int64_t left = a.M;; left -= most) {
        a.M = std::min(left, most);
        const dim3 grid(unsigned(ceil_div(a.N, 16)), unsigned(ceil_div(a.M, 8 * NT)));
        if (vec) gemm_i8_rows_kernel<TY, NT, true><<<grid, 256, 0, s>>>(a);
        else gemm_i8_rows_kernel<TY, NT, false><<<grid, 256, 0, s>>>(a);
        const int rc = check_launch();
        if (rc != REPOPS_OK || left <= most) return rc;
        if (a.A) a.A += most * a.lda;                          // null without k
        a.sa += most;
        a.C = static_cast<uint8_t *>(a.C) + most * a.ldc * int64_t(storage_size(TY));
    }
}

template <int TY>
int launch_rows(const I8Args &a, cudaStream_t s) {
    if (a.M <= 2) {
        // channels a warp: as many as leave 16 warps an SM
        const int64_t warps = int64_t(sm_count()) * 16;
        if (a.N >= 4 * warps) return launch_dot_r<TY, 4>(a, s);
        if (a.N >= 2 * warps) return launch_dot_r<TY, 2>(a, s);
        return launch_dot_r<TY, 1>(a, s);
    }
    if (a.M <= 8) return launch_rows_nt<TY, 1>(a, s);
    if (a.M <= 16) return launch_rows_nt<TY, 2>(a, s);
    if (a.M <= 32) return launch_rows_nt<TY, 4>(a, s);
    return launch_rows_nt<TY, 8>(a, s);
}

// A 2-D map of `rows` rows of `inner` values at pitch `ld`, a box of box_rows
// rows of 128 bytes under the 128-byte swizzle.
bool make_map(CUtensorMap *map, CUtensorMapDataType type, unsigned size, const void *base, int64_t inner, int64_t rows,
              int64_t ld, int box_inner, int box_rows) {
    gemm::EncodeTiledFn enc = gemm::tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(rows)}, strides[1] = {cuuint64_t(ld) * size};
    const cuuint32_t box[2] = {cuuint32_t(box_inner), cuuint32_t(box_rows)}, estr[2] = {1u, 1u};
    return enc(map, type, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The widened tokens as 64-k blocks: a box is BT tokens of two blocks, each with
// rows of 128 bytes under the 128-byte swizzle.
bool make_token_map(CUtensorMap *map, const __half *base, int64_t M, int64_t Kp, int box_rows) {
    gemm::EncodeTiledFn enc = gemm::tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {64u, cuuint64_t(M), cuuint64_t(Kp / 64)}, strides[2] = {cuuint64_t(Kp) * 2u, 128u};
    const cuuint32_t box[3] = {64u, cuuint32_t(box_rows), 2u}, estr[3] = {1u, 1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int TY, int BT>
int launch_stream(const I8Args &a, __half *tokens, int8_t *copy, cudaStream_t s) {
    using T = StreamCfg<BT>;
    const int64_t Kp = stream_k(a.K);
    const StreamMap sm = stream_map(a.M, a.N, a.K);
    // bytes that a 16-byte unit brings along behind K meet the tokens' zeros there
    const bool in_place = read_in_place(a.B, a.ldb), vec = operand_vec(a.A, a.lda);
    CUtensorMap mt, mw;
    if (!make_token_map(&mt, tokens, a.M * sm.copies, Kp, BT) ||
        !(in_place ? make_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.B, a.K, a.N, a.ldb, kStreamK, BM)
                   : make_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, copy, Kp, a.N, Kp, kStreamK, BM)))
        return REPOPS_ERR_UNSUPPORTED;
    unsigned *status = nullptr;
    int rc = status_word_address(&status);
    if (rc != REPOPS_OK) return rc;
    auto kern = gemm_i8_stream_kernel<TY, BT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
    if (e != cudaSuccess) return set_cuda_error(e);
    // nothing has been launched so far: from here on only a launch can fail
    const int64_t items = std::max(a.M * (Kp / 8), in_place ? int64_t(0) : a.N * (Kp / 16));
    const unsigned grid = unsigned(std::min<int64_t>(ceil_div(items, 512), int64_t(sm_count()) * 32));
    auto prep = in_place ? vec ? stream_prepare_kernel<true, false> : stream_prepare_kernel<false, false>
                         : vec ? stream_prepare_kernel<true, true> : stream_prepare_kernel<false, true>;
    prep<<<grid, 256, 0, s>>>(a, Kp, sm.copies, tokens, copy);
    rc = check_launch();
    if (rc != REPOPS_OK) return rc;
    constexpr unsigned csize = TY == REPOPS_TYPE_F32 ? 4u : 2u;
    const int c_vec = reinterpret_cast<uintptr_t>(a.C) % (4 * csize) == 0 && a.ldc % 4 == 0;
    const unsigned ctas = unsigned(sm.parts > 1 ? sm.tiles * sm.parts : std::min(sm.tiles, sm_count()));
    return launch_behind_cluster(kern, dim3(ctas), unsigned(sm.parts), kStreamThreads, T::SMEM, s, mt, mw, a, sm,
                                 int(in_place), c_vec, status);
}

template <int TY>
int launch_pair(const I8Args &a, __half *ws, cudaStream_t s) {
    using T = PairCfg;
    const int64_t Kp = padded_k(a.K);
    constexpr CUtensorMapDataType F16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap ma, mb, mc;
    if (!make_map(&ma, F16, 2, ws, Kp, a.M, Kp, BK, BM) || !make_map(&mb, F16, 2, ws + a.M * Kp, Kp, a.N, Kp, BK, T::B_ROWS))
        return REPOPS_ERR_UNSUPPORTED;
    // C by TMA where its rows start on 16 bytes and end on them: a store clips at
    // C's edge in units of 16 bytes, and what is behind a row is not C's
    constexpr unsigned csize = TY == REPOPS_TYPE_F32 ? 4u : 2u;
    constexpr CUtensorMapDataType ctype = TY == REPOPS_TYPE_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                          : TY == REPOPS_TYPE_F16 ? F16
                                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    constexpr int wide = 128 / int(csize);                             // columns of a stored block
    const int c_tma = reinterpret_cast<uintptr_t>(a.C) % 16 == 0 && uint64_t(a.ldc) * csize % 16 == 0 &&
                      uint64_t(a.N) * csize % 16 == 0 &&
                      a.ldc < (int64_t(1) << 37) && make_map(&mc, ctype, csize, a.C, a.N, a.M, a.ldc, wide, 32);
    if (!c_tma) mc = ma;
    unsigned *status = nullptr;
    int rc = status_word_address(&status);
    if (rc != REPOPS_OK) return rc;
    auto kern = gemm_i8_pair_kernel<TY>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
    if (e != cudaSuccess) return set_cuda_error(e);
    // nothing has been launched so far: from here on only a launch can fail
    const int64_t items = (a.M + a.N) * (Kp / 8);
    const unsigned wgrid = unsigned(std::min<int64_t>(ceil_div(items, 512), int64_t(sm_count()) * 32));
    if (operand_vec(a.A, a.lda) && operand_vec(a.B, a.ldb)) widen_kernel<true><<<wgrid, 256, 0, s>>>(a, Kp, ws);
    else widen_kernel<false><<<wgrid, 256, 0, s>>>(a, Kp, ws);
    rc = check_launch();
    if (rc != REPOPS_OK) return rc;
    const TileMap tm{int(ceil_div(a.M, 2 * BM)), int(ceil_div(a.N, T::BN)), 8};
    const int64_t tiles = int64_t(tm.tiles_m) * tm.tiles_n;
    return launch_behind(kern, dim3(unsigned(std::min<int64_t>(tiles, sm_count() / 2) * 2)), kPairThreads,
                         T::SMEM, s, ma, mb, mc, a, tm, int(Kp / BK), c_tma, status);
}

template <int TY>
int run_i8(int cfg, const I8Args &a, __half *ws, int8_t *copy, cudaStream_t s) {
    switch (cfg) {
        case CFG_ROWS: return launch_rows<TY>(a, s);
        case CFG_PAIR: return launch_pair<TY>(a, ws, s);
        default: return stream_tokens(a.M) == 64 ? launch_stream<TY, 64>(a, ws, copy, s) : launch_stream<TY, 128>(a, ws, copy, s);
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
    config = run_config(config, M, N, K);
    return config == CFG_ROWS ? 0 : config == CFG_PAIR ? pair_workspace(M, N, K) : stream_workspace(M, K);
}

extern "C" uint64_t repops_gemm_i8_operand_workspace_bytes(int config, int64_t M, int64_t N, int64_t K, const int8_t *B,
                                                           int64_t ldb) {
    return repops_gemm_i8_workspace_bytes(config, M, N, K) +
           (run_config(config, M, N, K) == CFG_TILES && !read_in_place(B, ldb) ? stream_copy_bytes(N, K) : 0u);
}

extern "C" int repops_gemm_i8(int config, int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda,
                              const float *a_scale, const int8_t *B, int64_t ldb, const float *b_scale,
                              const float *bias, void *C, int typeC, int64_t ldc, void *ws, uint64_t ws_bytes,
                              cudaStream_t stream) {
    if (M < 0 || N < 0 || K < 0 || !known_storage(typeC) || config < CFG_AUTO || config >= CFG_COUNT)
        return REPOPS_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return REPOPS_OK;
    if (K > kMaxK || M > INT32_MAX || N > INT32_MAX) return REPOPS_ERR_UNSUPPORTED;
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
    if (ceil_div(M, BM) * ceil_div(N, 16) > INT32_MAX / 2) return REPOPS_ERR_UNSUPPORTED;     // tile indices are 32-bit
    // scratch: `need` bytes from the caller or the pool, a copy of B (where one is
    // made) behind them where the caller's are that long, else from the pool
    const uint64_t need = repops_gemm_i8_workspace_bytes(config, M, N, K);
    const uint64_t all = repops_gemm_i8_operand_workspace_bytes(config, M, N, K, B, ldb);
    if (ws && need > 0) {
        if (ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 16 != 0) return REPOPS_ERR_INVALID_ARG;
        const uint64_t used = ws_bytes >= all ? all : need;
        if (ranges_overlap(ws, used, A, ab) || ranges_overlap(ws, used, B, bb) || ranges_overlap(ws, used, C, cb) ||
            ranges_overlap(ws, used, a_scale, sab) || ranges_overlap(ws, used, b_scale, sbb) ||
            (bias && ranges_overlap(ws, used, bias, sbb)))
            return REPOPS_ERR_ALIAS;
    }
    const uint64_t pool = !ws ? all : ws_bytes >= all ? 0 : all - need;
    void *own = nullptr;
    if (pool > 0 && scratch_malloc(&own, size_t(pool), stream) != cudaSuccess) {
        cudaGetLastError();
        return REPOPS_ERR_ALLOC;
    }
    __half *wide = static_cast<__half *>(ws ? ws : own);
    int8_t *copy = ws && own ? static_cast<int8_t *>(own) : reinterpret_cast<int8_t *>(wide + need / 2);
    I8Args a{{}, M, N, K, A, B, lda, ldb, a_scale, b_scale, bias, C, ldc, A + ab, B + bb};
    a.reads_words(A, ab);
    a.reads_words(B, bb);
    a.reads(a_scale, sab);
    a.reads(b_scale, sbb);
    a.reads(bias, sbb);
    a.writes(C, cb);
    a.writes(wide, need);
    a.writes(copy, all - need);
    int rc = a.arm();
    if (rc == REPOPS_OK)
        rc = typeC == REPOPS_TYPE_F32   ? run_i8<REPOPS_TYPE_F32>(config, a, wide, copy, stream)
             : typeC == REPOPS_TYPE_F16 ? run_i8<REPOPS_TYPE_F16>(config, a, wide, copy, stream)
                                        : run_i8<REPOPS_TYPE_BF16>(config, a, wide, copy, stream);
    if (own) {
        const cudaError_t e = cudaFreeAsync(own, stream);
        if (rc == REPOPS_OK && e != cudaSuccess) rc = set_cuda_error(e);
    }
    return rc;
}
