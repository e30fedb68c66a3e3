// The 8-bit linear layer's row operators of include/gemm_scaled.h: quantisation
// and the root-mean-square norm with its gradient.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "gemm_scaled.h"
#include "ptx.cuh"
#include "rows.cuh"

using namespace psm;

namespace {

constexpr int GROUP = GEMM_SCALE_GROUP;
constexpr float LEAST = 0x1p-100f;  // least magnitude that a scale is made from

// ---------------------------------------------------------------- 8 bits
template <bool E5M2>
struct Fp8 {
    static constexpr float LARGEST = E5M2 ? 57344.f : 448.f;
    static constexpr __nv_fp8_interpretation_t KIND = E5M2 ? __NV_E5M2 : __NV_E4M3;
};

// The scale of a group whose largest magnitude is m, and what its elements are
// multiplied by.
template <bool E5M2>
__device__ __forceinline__ float scale_of(float m) { return __fdiv_rn(fmaxf(m, LEAST), Fp8<E5M2>::LARGEST); }
template <bool E5M2>
__device__ __forceinline__ float inverse_of(float m) { return __fdiv_rn(Fp8<E5M2>::LARGEST, fmaxf(m, LEAST)); }

// The eight 8-bit values nearest to x * L / m, from v = x * exact_inverse_of(m).
//
// x * fl(L / m) is within 2^-23 of x * L / m, which could lift a quotient off a border
// between two 8-bit values or onto the other side, and between 16-bit x and m
// quotients on a border are common (0.3 % of normal bf16 values).  But those that are not on
// a border t (5 bits) are 2^-16 away from it at least: x L / m - t is a whole multiple
// of 1 / m over t of 5 bits and m of 11.  So the product, made 2^-21 larger, is cut
// to 20 bits: that puts what belongs on a border back onto it, and moves nothing
// across one.  (NaN and infinity stay what they are.)
template <bool E5M2>
__device__ __forceinline__ float exact_inverse_of(float m) { return __fmul_rn(inverse_of<E5M2>(m), 1.f + 0x1p-21f); }

template <bool E5M2, bool EXACT>
__device__ __forceinline__ uint2 quantized(const float (&v)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t pair[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float2 x = make_float2(v[4 * h + 2 * j], v[4 * h + 2 * j + 1]);
            if constexpr (EXACT) x = make_float2(__uint_as_float(__float_as_uint(x.x) & ~15u), __uint_as_float(__float_as_uint(x.y) & ~15u));
            pair[j] = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, Fp8<E5M2>::KIND);
        }
        w[h] = pair[0] | (pair[1] << 16);
    }
    return make_uint2(w[0], w[1]);
}

template <bool E5M2>
__device__ __forceinline__ uint2 quantized(const float (&x)[8], float inverse) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(x[i], inverse);
    return quantized<E5M2, true>(v);
}

// L / d within 2^-40 as the sum of two fp32 values, the second by one step of Newton's
// method, for d of at least 2^-120 (infinite or NaN: NaN).
struct Inverse {
    float high, low;
};
template <bool E5M2>
__device__ __forceinline__ Inverse inverse_in_two(float d) {
    constexpr float L = Fp8<E5M2>::LARGEST;
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
    const float high = __fmul_rn(L, r);
    return {high, __fmul_rn(__fmaf_rn(-high, d, L), r)};
}

// scale_of by two products.  1 / L in two parts is within 2^-46, and m / L, a whole number of
// sevenths of a power of two, is 1 / 14 of fp32's last digit away from the middle between two
// fp32 values at least, so their sum is rounded as the quotient.  (Both parts are positive, so
// that an infinity stays one.)
template <bool E5M2>
__device__ __forceinline__ float scale_by_products(float m) {
    constexpr float L = Fp8<E5M2>::LARGEST, HIGH = 0x1.249248p-3f * (7.f / L), LOW = (float)(1. / L - (double)HIGH);
    static_assert(LOW > 0.f, "1 / 7 cut, not rounded");
    return __fmaf_rn(m, HIGH, __fmul_rn(m, LOW));
}

// The eight 8-bit values nearest to the quotients z * L / m, where m is the largest |z| of the
// group, for z = s * weight of two 16-bit values, exact in fp32.
//
// The product with L / m in two parts is the quotient with one rounding of 2^-24.  So one on a
// border between two 8-bit values stays on it, and one that is not does not get onto
// its other side.  bf16: nor onto it, as it is 2^-21 away at least (z L is a whole multiple of
// its last digit over z of 16 bits, t m of its over t of 5 bits and m of 16).  fp16 (z and m of 22
// bits): where it does, the sign of |z| L - t m, in two parts each, says from which side (not
// for m = NaN, of a group whose scale is not made from its largest).
template <typename T, bool E5M2>
__device__ __forceinline__ uint2 nearest(const float (&z)[8], Inverse in, float m) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmaf_rn(z[i], in.high, __fmul_rn(z[i], in.low));
    if constexpr (!std::is_same_v<T, __nv_bfloat16>) {
        constexpr uint32_t BELOW = E5M2 ? 0x1fffffu : 0xfffffu, HALF = BELOW / 2 + 1;  // fp32's digits after those of the type
        constexpr float L = Fp8<E5M2>::LARGEST, NORMAL = E5M2 ? 0x1p-14f : 0x1p-6f;    // the least value with a leading one
        bool close = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) close |= (__float_as_uint(v[i]) & BELOW) == HALF || fabsf(v[i]) < NORMAL;
        if (close)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // below NORMAL the steps are those of the 2^n above it
                const float a = fabsf(v[i]), shift = a < NORMAL ? NORMAL : 0.f;
                const float t = __uint_as_float((__float_as_uint(a + shift) & ~BELOW) | HALF) - shift;
                if (a == t) {
                    const float y = fabsf(z[i]), p = __fmul_rn(y, L), q = __fmul_rn(t, m);
                    const float d = (p - q) + (__fmaf_rn(y, L, -p) - __fmaf_rn(t, m, -q));
                    v[i] = copysignf(__uint_as_float(__float_as_uint(t) + (d > 0.f) - (d < 0.f)), v[i]);
                }
            }
    }
    return quantized<E5M2, false>(v);
}

// Elements h .. h + 7 of a row of n to memory; ALIGNED: all of them, at once.
template <bool ALIGNED>
__device__ __forceinline__ void store_quantized(uint8_t* row, int h, int n, uint2 q) {
    if constexpr (ALIGNED) {
        *reinterpret_cast<uint2*>(row + h) = q;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (h + i < n) row[h + i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
    }
}

// The same by all lanes of a warp, of which 16 in turn have the chunks of a group (`ok`:
// the row is there).  Off the grid these go through shared memory, where each word of
// the row is cut from two, and are stored 4 bytes a lane (us, element by element and so:
// 5003 x 2055 along the rows 21.3 / 18.3, the columns 29.0 / 21.1, both 45.1 / 32.0).
template <bool ALIGNED>
__device__ __forceinline__ void store_group(uint8_t* row, int h, int n, uint2 q, bool ok) {
    if constexpr (ALIGNED) {
        if (ok && h < n) *reinterpret_cast<uint2*>(row + h) = q;
    } else {
        __shared__ uint32_t buffer[16][34];
        const int lane = threadIdx.x & 15;
        uint32_t* mine = buffer[threadIdx.x >> 4];
        __syncwarp();  // what was stored before has been read
        mine[2 * lane] = q.x;
        mine[2 * lane + 1] = q.y;
        __syncwarp();
        uint8_t* at = row + h - 8 * lane;
        const int bytes = ok ? max(0, min(n - h + 8 * lane, GROUP)) : 0;
        const int head = min((int)(-reinterpret_cast<uintptr_t>(at) & 3), bytes);  // before the first whole word
        const int words = (bytes - head) >> 2, tail = head + 4 * words;
#pragma unroll
        for (int j = lane; j < 32; j += 16)  // (the second word of the last one is not used)
            if (j < words) *reinterpret_cast<uint32_t*>(at + head + 4 * j) = __funnelshift_r(mine[j], mine[j + 1], 8 * head);
        const uint8_t* own = reinterpret_cast<const uint8_t*>(mine);
        if (lane < head) at[lane] = own[lane];
        if (tail + lane < bytes) at[tail + lane] = own[tail + lane];
    }
}

template <bool ALIGNED>
__device__ __forceinline__ void store_16bit(uint16_t* row, int h, int n, const Chunk& c) {
    if constexpr (ALIGNED) {
        *reinterpret_cast<uint4*>(row + h) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (h + i < n) row[h + i] = (uint16_t)(c.w[i / 2] >> (16 * (i & 1)));
    }
}

// Elements h .. h + 7 of a row of n as fp32, zeros past its end.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void load_row(const uint16_t* row, int h, int n, float (&x)[8]) {
    unpack<T>(load_chunk<ALIGNED>(row, h, n), x);
    if constexpr (!ALIGNED)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (h + i >= n) x[i] = 0.f;
}

__device__ __forceinline__ float magnitude(const float (&x)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    return m;
}

// The largest over the 16 lanes that share a row's group.
__device__ __forceinline__ float over_half(float m) {
#pragma unroll
    for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// ---------------------------------------------------------------- quantisation
struct QuantizeArgs {
    const uint16_t* x;
    int64_t ldx, rows;
    int cols, row_groups;  // row_groups: groups of a row
    uint8_t* q;            // ROWS, or COLS / BLOCKS alone
    int64_t ldq;
    float* scales;
    uint8_t* q_cols;       // BOTH: the columns' form
    int64_t ldq_cols;
    float* scales_cols;
};

// Vectors along the rows (8192 x 4096 in 21.9 us, 4.7 TB/s; issue slots 69 % busy): 16 lanes a group, a block takes R rows and its 16 / R
// half-warps a row, U groups each.
template <typename T, bool E5M2, bool ALIGNED, int R, int U>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantizeArgs a) {
    const int half = threadIdx.x >> 4, lane = threadIdx.x & 15;
    constexpr int ACROSS = 16 / R;
    const int strips = (a.row_groups + ACROSS * U - 1) / (ACROSS * U);
    const int64_t row = (int64_t)(blockIdx.x / strips) * R + half % R;
    const int g0 = (blockIdx.x % strips) * ACROSS * U + half / R;
    grid_dependency_wait();
    grid_launch_dependents();
    float x[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = (g0 + u * ACROSS) * GROUP + lane * 8;
        if (row < a.rows && h < a.cols) load_row<T, ALIGNED>(a.x + row * a.ldx, h, a.cols, x[u]);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int g = g0 + u * ACROSS, h = g * GROUP + lane * 8;
        const float m = over_half(magnitude(x[u]));
        store_group<ALIGNED>(a.q + row * a.ldq, h, a.cols, quantized<E5M2>(x[u], exact_inverse_of<E5M2>(m)), row < a.rows);
        if (row < a.rows && h < a.cols && lane == 0) a.scales[(int64_t)g * a.rows + row] = scale_of<E5M2>(m);
    }
}

// Tiles of 128 x 128: vectors along the columns, a block, or vectors along both
// dimensions.  A thread has eight columns of eight rows, 16 apart, which stay in
// registers between the magnitudes and the output, so the matrix is read once.  Blocks an
// SM: bytes in flight against registers that spill.  us with 2, 3, 4: blocks of 14336 x 4096
// 40.8 / 35.1 / 33.4, columns of 8192 x 4096 25.2 / 23.9 / 23.3, both 39.8 / 44.7 / 48.8 (since,
// with a cheaper rounding, 31.1 at 5.7 TB/s, 21.7 and 36.5).  With both, latency: two blocks of 106
// registers a thread leave issue slots half empty.
template <typename T, bool E5M2, bool ALIGNED, int KIND, bool BOTH>
__global__ void __launch_bounds__(256, BOTH ? 2 : 4) quantize_tile_kernel(QuantizeArgs a) {
    __shared__ float part[8][GROUP];
    const int lane = threadIdx.x & 15, r = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const int64_t tile_row = blockIdx.x / a.row_groups;
    const int tile_col = blockIdx.x % a.row_groups;
    const int h = tile_col * GROUP + lane * 8;
    const int64_t row0 = tile_row * GROUP + r;
    grid_dependency_wait();
    grid_launch_dependents();
    Chunk c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = row0 + 16 * i;
        if (row < a.rows && h < a.cols) c[i] = load_chunk<ALIGNED>(a.x + row * a.ldx, h, a.cols);
        else c[i] = Chunk{};
    }
    float col[8] = {};  // the largest magnitude of each of this thread's columns
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float x[8];
        unpack<T>(c[i], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!ALIGNED && h + j >= a.cols) x[j] = 0.f;
            col[j] = fmaxf(col[j], fabsf(x[j]));
        }
        if constexpr (BOTH) {
            const int64_t row = row0 + 16 * i;
            const float m = over_half(magnitude(x));
            store_group<ALIGNED>(a.q + row * a.ldq, h, a.cols, quantized<E5M2>(x, exact_inverse_of<E5M2>(m)), row < a.rows);
            if (row < a.rows && lane == 0) a.scales[(int64_t)tile_col * a.rows + row] = scale_of<E5M2>(m);
        }
    }
    if constexpr (KIND == GEMM_QUANTIZE_BLOCKS) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, col[j]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((threadIdx.x & 31) == 0) part[0][warp] = m;
        __syncthreads();
        m = part[0][threadIdx.x & 7];
#pragma unroll
        for (int o = 4; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (threadIdx.x == 0) a.scales[tile_row * a.row_groups + tile_col] = scale_of<E5M2>(m);
        const float inverse = exact_inverse_of<E5M2>(m);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t row = row0 + 16 * i;
            float x[8];
            unpack<T>(c[i], x);
            store_group<ALIGNED>(a.q + row * a.ldq, h, a.cols, quantized<E5M2>(x, inverse), row < a.rows);
        }
    } else {
        uint8_t* q = BOTH ? a.q_cols : a.q;
        const int64_t ldq = BOTH ? a.ldq_cols : a.ldq;
        float* scales = BOTH ? a.scales_cols : a.scales;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            col[j] = fmaxf(col[j], __shfl_xor_sync(0xffffffffu, col[j], 16));
            if ((threadIdx.x & 16) == 0) part[warp][lane * 8 + j] = col[j];
        }
        __syncthreads();
        if (threadIdx.x < GROUP) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, part[i][threadIdx.x]);
            const int at = tile_col * GROUP + threadIdx.x;
            if (at < a.cols) scales[tile_row * a.cols + at] = scale_of<E5M2>(m);
            part[0][threadIdx.x] = exact_inverse_of<E5M2>(m);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) col[j] = part[0][lane * 8 + j];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t row = row0 + 16 * i;
            float x[8];
            unpack<T>(c[i], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(x[j], col[j]);
            store_group<ALIGNED>(q + row * ldq, h, a.cols, quantized<E5M2, true>(x), row < a.rows);
        }
    }
}

// Whether rows of 16-bit inputs and 8-bit outputs can be taken in chunks of eight.
bool whole_chunks(int64_t cols, std::initializer_list<const void*> in, std::initializer_list<int64_t> ld_in,
                  std::initializer_list<const void*> out, std::initializer_list<int64_t> ld_out) {
    int64_t bits = cols * 2;
    for (const void* p : in) bits |= (int64_t)(uintptr_t)p;
    for (int64_t ld : ld_in) bits |= ld * 2;
    for (const void* p : out) bits |= (int64_t)(uintptr_t)p * 2;
    for (int64_t ld : ld_out) bits |= ld * 2;
    return (bits & 15) == 0;
}

template <typename T, bool E5M2, bool ALIGNED>
gemm_status_t quantize_v(int kind, bool both, const QuantizeArgs& a, gemm_stream_t stream) {
    if (kind == GEMM_QUANTIZE_ROWS && !both) {
        const bool few = a.rows < 8;
        const int64_t grid = few ? a.rows * cdiv(a.row_groups, 16) : cdiv(a.rows, 8) * cdiv(a.row_groups, 8);
        if (grid > MAX_INDEX) return GEMM_ERR_UNSUPPORTED;
        return launch(few ? quantize_rows_kernel<T, E5M2, ALIGNED, 1, 1> : quantize_rows_kernel<T, E5M2, ALIGNED, 8, 4>,
                      dim3((unsigned)grid), dim3(256), 0, stream, a);
    }
    const int64_t grid = cdiv(a.rows, GROUP) * a.row_groups;
    if (grid > MAX_INDEX) return GEMM_ERR_UNSUPPORTED;
    auto* fn = both                             ? quantize_tile_kernel<T, E5M2, ALIGNED, GEMM_QUANTIZE_COLS, true>
               : kind == GEMM_QUANTIZE_COLS     ? quantize_tile_kernel<T, E5M2, ALIGNED, GEMM_QUANTIZE_COLS, false>
                                                : quantize_tile_kernel<T, E5M2, ALIGNED, GEMM_QUANTIZE_BLOCKS, false>;
    return launch(fn, dim3((unsigned)grid), dim3(256), 0, stream, a);
}

template <typename T, bool E5M2>
gemm_status_t quantize(int kind, bool both, const QuantizeArgs& a, gemm_stream_t stream) {
    const bool al = both ? whole_chunks(a.cols, {a.x}, {a.ldx}, {a.q, a.q_cols}, {a.ldq, a.ldq_cols})
                         : whole_chunks(a.cols, {a.x}, {a.ldx}, {a.q}, {a.ldq});
    return (al ? quantize_v<T, E5M2, true> : quantize_v<T, E5M2, false>)(kind, both, a, stream);
}

gemm_status_t quantize_any(int kind, bool both, const QuantizeArgs& a, int dtype, int type, gemm_stream_t stream) {
    auto* fn = dtype == GEMM_BF16 ? (type == GEMM_E5M2 ? quantize<__nv_bfloat16, true> : quantize<__nv_bfloat16, false>)
                                  : (type == GEMM_E5M2 ? quantize<__half, true> : quantize<__half, false>);
    return fn(kind, both, a, stream);
}

bool bad_types(int dtype, int type) {
    return (dtype != GEMM_F16 && dtype != GEMM_BF16) || (type != GEMM_E4M3 && type != GEMM_E5M2);
}

// ---------------------------------------------------------------- norm
struct NormArgs {
    const uint16_t *x, *residual, *weight;
    int64_t ldx, ldres, rows;
    int hidden;
    float eps;
    uint16_t *sum, *y;
    int64_t ldsum, ldy;
    uint8_t* q;
    int64_t ldq;
    float *scales, *rstd;
};

// Sum over the threads of a row (threadIdx.y); `part` has room for a float a warp
// of the block.
__device__ __forceinline__ float over_row(float v, float* part) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.y * warps + warp] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = lane < warps ? part[threadIdx.y * warps + lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Elements h .. h + 7 of a row of n, zeros past its end.
template <bool ALIGNED, bool ONCE = true>
__device__ __forceinline__ Chunk load_masked(const uint16_t* row, int h, int n) {
    if (h >= n) return Chunk{};
    if constexpr (ALIGNED && !ONCE) return load_word<false>(row + h);
    Chunk c = load_chunk<ALIGNED>(row, h, n);
    if constexpr (!ALIGNED)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (h + i >= n) c.w[i / 2] &= i & 1 ? 0x0000ffffu : 0xffff0000u;
    return c;
}

// A row of `blockDim.x` threads, V chunks each, strided by blockDim.x, so that
// 16 lanes have a group.  Bound by instructions (issue slots 70 % busy with 8-bit output) as much as
// by memory.  The row stays in registers between the
// sum and the output, and so does the weight over all the rows that a block takes
// (every gridDim.x x blockDim.y th); AHEAD: the next row is on its way while this
// one is summed and written, which keeps reads in flight over the barrier.  8192 rows of
// 4096 with residual and 8-bit output: 45.3 us, 5.2 TB/s (59 with a row a block and no
// row ahead).  Q: with 8-bit output; without it, kernels of their own have registers to spare
// (us, in one kernel and so: 16-bit output of 8192 x 4096 30.4 / 28.1).
//
// 8-bit values from y by one product with the rounded inverse, some of them on the other side of
// a border: 44.4 us; from s * weight in two parts, but the scales and inverses by divisions: 47.7.
template <typename T, bool Q, bool E5M2, bool ALIGNED, int V, bool AHEAD, int THREADS, int RESIDENT>
__global__ void __launch_bounds__(THREADS, RESIDENT) norm_kernel(NormArgs a) {
    __shared__ float part[2][32];
    const int n = a.hidden;
    grid_dependency_wait();
    grid_launch_dependents();
    auto added = [&](const Chunk& x, const Chunk& r) {
        float f[8], g[8];
        unpack<T>(x, f);
        unpack<T>(r, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += g[i];
        return pack<T>(f);
    };
    // without AHEAD registers are short: the sum is made at once, the weight read when used
    Chunk w[AHEAD ? V : 1], x[V], r[AHEAD ? V : 1];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int h = (v * blockDim.x + threadIdx.x) * 8;
            x[v] = Chunk{};
            if (AHEAD) r[v] = Chunk{};
            if (row >= a.rows) continue;
            x[v] = load_masked<ALIGNED>(a.x + row * a.ldx, h, n);
            if (!a.residual) continue;
            const Chunk c = load_masked<ALIGNED>(a.residual + row * a.ldres, h, n);
            if (AHEAD) r[v] = c;
            else x[v] = added(x[v], c);
        }
    };
    int64_t first = (int64_t)blockIdx.x * blockDim.y;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    load(first + threadIdx.y);
    if (AHEAD)
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] = load_masked<ALIGNED, false>(a.weight, (v * blockDim.x + threadIdx.x) * 8, n);
    int turn = 0;
#pragma unroll 1
    for (; first < a.rows; first += step, turn ^= 1) {
        const int64_t row = first + threadIdx.y;
        const bool in = row < a.rows;
        Chunk s[V];
        float square = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = AHEAD && a.residual ? added(x[v], r[v]) : x[v];
            float f[8];
            unpack<T>(s[v], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) square = fmaf(f[i], f[i], square);
        }
        if (AHEAD) load(row + step);
        square = over_row(square, part[turn]);
        const float rstd = __frsqrt_rn(__fdiv_rn(square, (float)n) + a.eps);
        if (in && threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
        // the least s * weight that a scale is made from: that of LEAST, while fp32 holds it exactly
        [[maybe_unused]] const float least = fminf(fmaxf(__fdiv_rn(LEAST, rstd), 0x1p-120f), 0x1p100f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int h = (v * blockDim.x + threadIdx.x) * 8;
            const bool here = in && h < n;
            float f[8], g[8];
            unpack<T>(s[v], f);
            unpack<T>(AHEAD ? w[v] : load_masked<ALIGNED, false>(a.weight, h, n), g);
            if constexpr (!Q) {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = f[i] * rstd * g[i];
                if (here) {
                    if (a.sum) store_16bit<ALIGNED>(a.sum + row * a.ldsum, h, n, s[v]);
                    if (a.y) store_16bit<ALIGNED>(a.y + row * a.ldy, h, n, pack<T>(f));
                }
            } else {
                if (here) {
                    if (a.sum) store_16bit<ALIGNED>(a.sum + row * a.ldsum, h, n, s[v]);
                    if (a.y) {
                        float y[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = f[i] * rstd * g[i];
                        store_16bit<ALIGNED>(a.y + row * a.ldy, h, n, pack<T>(y));
                    }
                }
                // The row's factor cancels from y / m, so the values are made from z = s * weight, which
                // fp32 holds exactly.  (Made from y, its two roundings would decide for quotients
                // on a border, which are common between products of 16-bit values.)
                float z[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = f[i] * g[i];
                const float largest = over_half(magnitude(z)), top = fmaxf(largest, least), m = top * rstd;
                Inverse inverse = inverse_in_two<E5M2>(top);
                inverse.low += m * 0.f;  // NaN where m is infinite or NaN
                if (here) {
                    store_quantized<ALIGNED>(a.q + row * a.ldq, h, n, nearest<T, E5M2>(z, inverse, largest >= least ? top : NAN));
                    if ((threadIdx.x & 15) == 0) a.scales[(int64_t)(h / GROUP) * a.rows + row] = scale_by_products<E5M2>(fmaxf(m, LEAST));
                }
            }
        }
        if (!AHEAD) load(row + step);
    }
}

struct NormGradArgs {
    const uint16_t *dy, *s, *weight, *dsum;
    const float* rstd;
    int64_t lddy, lds, lddsum, rows, lddx;
    int hidden;
    uint16_t* dx;
    float* part;  // gridDim.x x hidden, or null
};

// As norm_kernel, a row a block: a thread has the same columns of every row and
// sums their dweight in registers.  16384 rows of 4096: 91 us with the sum of the
// blocks' parts, 5.9 TB/s (148 without the row ahead).
template <typename T, bool ALIGNED, int V, bool AHEAD, int THREADS, int RESIDENT>
__global__ void __launch_bounds__(THREADS, RESIDENT) norm_grad_kernel(NormGradArgs a) {
    __shared__ float part[2][32];
    const int n = a.hidden;
    grid_dependency_wait();
    grid_launch_dependents();
    Chunk w[AHEAD ? V : 1], dy[V], s[V], d[AHEAD ? V : 1];
    auto weight = [&](int v) { return load_masked<ALIGNED, false>(a.weight, (v * blockDim.x + threadIdx.x) * 8, n); };
    float rstd = 0.f;
    auto load = [&](int64_t row) {
        if (row >= a.rows) return;
        rstd = a.rstd[row];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int h = (v * blockDim.x + threadIdx.x) * 8;
            dy[v] = load_masked<ALIGNED>(a.dy + row * a.lddy, h, n);
            s[v] = load_masked<ALIGNED>(a.s + row * a.lds, h, n);
            if (AHEAD) d[v] = a.dsum ? load_masked<ALIGNED>(a.dsum + row * a.lddsum, h, n) : Chunk{};
        }
    };
    load(blockIdx.x);
    if (AHEAD)
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] = weight(v);
    float dw[V][8] = {};
    int turn = 0;
#pragma unroll 1
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const float scale = rstd;
        Chunk p[V], q[V], e[AHEAD ? V : 1];
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float g[8], f[8], c[8];
            unpack<T>(dy[v], g);
            unpack<T>(s[v], f);
            unpack<T>(AHEAD ? w[v] : weight(v), c);
            p[v] = dy[v];
            q[v] = s[v];
            if (AHEAD) e[v] = d[v];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = g[i] * (f[i] * scale);
                dw[v][i] += x;
                dot = fmaf(x, c[i], dot);
            }
        }
        if (AHEAD) load(row + gridDim.x);
        const float mean = __fdiv_rn(over_row(dot, part[turn]), (float)n);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int h = (v * blockDim.x + threadIdx.x) * 8;
            if (h >= n) continue;
            float g[8], f[8], c[8], b[8];
            unpack<T>(p[v], g);
            unpack<T>(q[v], f);
            unpack<T>(AHEAD ? w[v] : weight(v), c);
            unpack<T>(AHEAD ? e[v] : a.dsum ? load_masked<ALIGNED>(a.dsum + row * a.lddsum, h, n) : Chunk{}, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = scale * (c[i] * g[i] - (f[i] * scale) * mean) + b[i];
            store_16bit<ALIGNED>(a.dx + row * a.lddx, h, n, pack<T>(g));
        }
        if (!AHEAD) load(row + gridDim.x);
    }
    if (a.part)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int h = (v * blockDim.x + threadIdx.x) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (h + i < n) a.part[(int64_t)blockIdx.x * n + h + i] = dw[v][i];
        }
}

// dweight = the sum of the blocks' parts: 32 columns a block, its warps take the
// parts in turn.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* part, int blocks, int n, float* dweight) {
    __shared__ float sums[32][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    float sum = 0.f;
    if (col < n)
        for (int b = warp; b < blocks; b += 32) sum += part[(int64_t)b * n + col];
    sums[warp][threadIdx.x & 31] = sum;
    __syncthreads();
    if (warp == 0 && col < n) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) sum += sums[i][threadIdx.x];
        dweight[col] = sum;
    }
}

// Threads of a row with v chunks each, and rows of a block.
dim3 norm_block(int64_t hidden, int v) {
    const int64_t chunks = cdiv(hidden, 8);
    const unsigned width = (unsigned)(std::max<int64_t>(cdiv(cdiv(chunks, v), 32), 1) * 32);
    return dim3(width, width < 256 ? 256 / width : 1, 1);
}

constexpr int SMS = 152;
// Blocks of 256 an SM: more bytes in flight against registers that spill.  us with 2, 3, 4:
// norm of 8192 rows of 4096 45.0 / 44.4 / 48.1, 16384 of 1024 31.6 / 24.6 / 25.6; gradient
// with 1, 2, 3: 16384 rows of 4096 116 / 91 / 116, of 1024 48 / 33 / 32.
// Norms of short rows without 8-bit output have the registers for four: 16384 of 1024 19.7 / 18.4
// with 3, 4; 5003 of 1001 22.5 / 17.8.
constexpr int NORM_RESIDENT = 3, GRAD_RESIDENT = 2;
// Blocks of `threads` that are resident at once where `resident` of `most` are.
int64_t resident_blocks(int64_t threads, int most, int resident) {
    return SMS * std::max<int64_t>(1, most * resident / threads);
}

template <typename T, bool Q, bool E5M2, bool ALIGNED>
gemm_status_t norm_v(const NormArgs& a, gemm_stream_t stream) {
    const int64_t chunks = cdiv(a.hidden, 8);
    auto run = [&](void (*fn)(NormArgs), int v, int most, int resident) {
        const dim3 block = norm_block(a.hidden, v);
        const int64_t grid = std::min(cdiv(a.rows, block.y), resident_blocks(block.x * block.y, most, resident));
        return launch(fn, dim3((unsigned)grid), block, 0, stream, a);
    };
    if (chunks <= 256) return run(norm_kernel<T, Q, E5M2, ALIGNED, 1, true, 256, Q ? NORM_RESIDENT : 4>, 1, 256, Q ? NORM_RESIDENT : 4);
    if (chunks <= 512) return run(norm_kernel<T, Q, E5M2, ALIGNED, 2, true, 256, NORM_RESIDENT>, 2, 256, NORM_RESIDENT);
    if (chunks <= 1024) return run(norm_kernel<T, Q, E5M2, ALIGNED, 2, true, 512, 2>, 2, 512, 2);
    if (chunks <= 2048) return run(norm_kernel<T, Q, E5M2, ALIGNED, 2, true, 1024, 1>, 2, 1024, 1);
    return run(norm_kernel<T, Q, E5M2, ALIGNED, 4, false, 1024, 1>, 4, 1024, 1);
}

template <typename T, bool Q, bool E5M2>
gemm_status_t norm(const NormArgs& a, bool aligned, gemm_stream_t stream) {
    return (aligned ? norm_v<T, Q, E5M2, true> : norm_v<T, Q, E5M2, false>)(a, stream);
}

template <typename T>
gemm_status_t norm_any(const NormArgs& a, bool aligned, int type, gemm_stream_t stream) {
    return (!a.q ? norm<T, false, false> : type == GEMM_E5M2 ? norm<T, true, true> : norm<T, true, false>)(a, aligned, stream);
}

// How the gradient of rows of `hidden` is launched.
struct GradShape {
    int v, most, resident;
    int64_t threads, blocks;
};

GradShape grad_shape(int64_t rows, int64_t hidden) {
    const int64_t chunks = cdiv(hidden, 8);
    GradShape s = chunks <= 256 ? GradShape{1, 256, GRAD_RESIDENT} : chunks <= 512 ? GradShape{2, 256, GRAD_RESIDENT} : chunks <= 1024 ? GradShape{2, 512, 1}
                : chunks <= 2048 ? GradShape{4, 512, 1} : GradShape{4, 1024, 1};
    s.threads = norm_block(hidden, s.v).x;
    s.blocks = std::min(rows, resident_blocks(s.threads, s.most, s.resident));
    return s;
}

template <typename T, bool ALIGNED>
gemm_status_t norm_grad_v(const NormGradArgs& a, float* dweight, gemm_stream_t stream) {
    const GradShape s = grad_shape(a.rows, a.hidden);
    auto* fn = s.v == 1       ? norm_grad_kernel<T, ALIGNED, 1, true, 256, GRAD_RESIDENT>
               : s.v == 2     ? (s.most == 256 ? norm_grad_kernel<T, ALIGNED, 2, true, 256, GRAD_RESIDENT> : norm_grad_kernel<T, ALIGNED, 2, true, 512, 1>)
               : s.most == 512 ? norm_grad_kernel<T, ALIGNED, 4, false, 512, 1>
                               : norm_grad_kernel<T, ALIGNED, 4, false, 1024, 1>;
    const gemm_status_t st = launch(fn, dim3((unsigned)s.blocks), dim3((unsigned)s.threads), 0, stream, a);
    if (st != GEMM_OK || !dweight) return st;
    return launch(norm_weight_kernel, dim3((unsigned)cdiv(a.hidden, 32)), dim3(1024), 0, stream, a.part, (int)s.blocks, a.hidden, dweight);
}

template <typename T>
gemm_status_t norm_grad(const NormGradArgs& a, bool aligned, float* dweight, gemm_stream_t stream) {
    return (aligned ? norm_grad_v<T, true> : norm_grad_v<T, false>)(a, dweight, stream);
}

gemm_status_t check_norm(int64_t rows, int64_t hidden) {
    if (rows < 0 || hidden < 0) return GEMM_ERR_INVALID_ARG;
    return rows > MAX_INDEX || hidden > GEMM_NORM_MAX_HIDDEN ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t gemm_scaled_quantize(gemm_quantize_t kind, const void* x, int64_t ldx, int64_t rows,
                                   int64_t cols, gemm_dtype_t dtype, gemm_fp8_t type, void* q,
                                   int64_t ldq, float* scales, gemm_stream_t stream) {
    if ((kind != GEMM_QUANTIZE_ROWS && kind != GEMM_QUANTIZE_COLS && kind != GEMM_QUANTIZE_BLOCKS) ||
        bad_types(dtype, type) || rows < 0 || cols < 0 || ldx < cols || ldq < cols)
        return GEMM_ERR_INVALID_ARG;
    const bool empty = rows == 0 || cols == 0;
    if (!empty && (!x || !q || !scales)) return GEMM_ERR_INVALID_ARG;
    if (rows > MAX_INDEX || cols > MAX_INDEX || misaligned(x, 2) || misaligned(scales, 4)) return GEMM_ERR_UNSUPPORTED;
    if (empty) return GEMM_OK;
    QuantizeArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.ldx = ldx;
    a.rows = rows;
    a.cols = (int)cols;
    a.row_groups = (int)cdiv(cols, GROUP);
    a.q = static_cast<uint8_t*>(q);
    a.ldq = ldq;
    a.scales = scales;
    return quantize_any(kind, false, a, dtype, type, stream);
}

gemm_status_t gemm_scaled_quantize_both(const void* x, int64_t ldx, int64_t rows, int64_t cols,
                                        gemm_dtype_t dtype, gemm_fp8_t type, void* q_rows,
                                        int64_t ldq_rows, float* scales_rows, void* q_cols,
                                        int64_t ldq_cols, float* scales_cols, gemm_stream_t stream) {
    if (bad_types(dtype, type) || rows < 0 || cols < 0 || ldx < cols || ldq_rows < cols || ldq_cols < cols)
        return GEMM_ERR_INVALID_ARG;
    const bool empty = rows == 0 || cols == 0;
    if (!empty && (!x || !q_rows || !scales_rows || !q_cols || !scales_cols)) return GEMM_ERR_INVALID_ARG;
    if (rows > MAX_INDEX || cols > MAX_INDEX || misaligned(x, 2) || misaligned(scales_rows, 4) || misaligned(scales_cols, 4))
        return GEMM_ERR_UNSUPPORTED;
    if (empty) return GEMM_OK;
    QuantizeArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.ldx = ldx;
    a.rows = rows;
    a.cols = (int)cols;
    a.row_groups = (int)cdiv(cols, GROUP);
    a.q = static_cast<uint8_t*>(q_rows);
    a.ldq = ldq_rows;
    a.scales = scales_rows;
    a.q_cols = static_cast<uint8_t*>(q_cols);
    a.ldq_cols = ldq_cols;
    a.scales_cols = scales_cols;
    return quantize_any(GEMM_QUANTIZE_COLS, true, a, dtype, type, stream);
}

gemm_status_t gemm_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldres,
                            const void* weight, float eps, int64_t rows, int64_t hidden,
                            gemm_dtype_t dtype, void* sum, int64_t ldsum, void* y, int64_t ldy,
                            void* q, int64_t ldq, gemm_fp8_t type, float* scales, float* rstd,
                            gemm_stream_t stream) {
    const gemm_status_t st = check_norm(rows, hidden);
    if (st == GEMM_ERR_INVALID_ARG || bad_types(dtype, type) || !(eps >= 0.f) || ldx < hidden ||
        (residual && ldres < hidden) || (sum && (ldsum < hidden || !residual)) || (y && ldy < hidden) ||
        (q && ldq < hidden) || (!q != !scales))
        return GEMM_ERR_INVALID_ARG;
    const bool empty = rows == 0 || hidden == 0;
    if (!empty && (!x || !weight || (!y && !q))) return GEMM_ERR_INVALID_ARG;
    if (st != GEMM_OK) return st;
    if (misaligned(x, 2) || misaligned(residual, 2) || misaligned(weight, 2) || misaligned(sum, 2) || misaligned(y, 2) ||
        misaligned(scales, 4) || misaligned(rstd, 4))
        return GEMM_ERR_UNSUPPORTED;
    if (empty) return GEMM_OK;
    NormArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.residual = static_cast<const uint16_t*>(residual);
    a.weight = static_cast<const uint16_t*>(weight);
    a.ldx = ldx;
    a.ldres = residual ? ldres : 0;
    a.rows = rows;
    a.hidden = (int)hidden;
    a.eps = eps;
    a.sum = static_cast<uint16_t*>(sum);
    a.y = static_cast<uint16_t*>(y);
    a.ldsum = sum ? ldsum : 0;
    a.ldy = y ? ldy : 0;
    a.q = static_cast<uint8_t*>(q);
    a.ldq = q ? ldq : 0;
    a.scales = scales;
    a.rstd = rstd;
    const bool al = whole_chunks(hidden, {x, residual, weight, sum, y}, {ldx, a.ldres, a.ldsum, a.ldy}, {q}, {a.ldq});
    return (dtype == GEMM_BF16 ? norm_any<__nv_bfloat16> : norm_any<__half>)(a, al, type, stream);
}

gemm_status_t gemm_rms_norm_grad_workspace_size(int64_t rows, int64_t hidden, size_t* bytes) {
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = check_norm(rows, hidden);
    if (st != GEMM_OK) return st;
    *bytes = rows == 0 || hidden == 0 ? 0 : (size_t)grad_shape(rows, hidden).blocks * (size_t)hidden * sizeof(float);
    return GEMM_OK;
}

gemm_status_t gemm_rms_norm_grad(const void* dy, int64_t lddy, const void* s, int64_t lds,
                                 const void* weight, const float* rstd, const void* dsum,
                                 int64_t lddsum, int64_t rows, int64_t hidden, gemm_dtype_t dtype,
                                 void* dx, int64_t lddx, float* dweight, void* workspace,
                                 gemm_stream_t stream) {
    const gemm_status_t st = check_norm(rows, hidden);
    if (st == GEMM_ERR_INVALID_ARG || bad_types(dtype, GEMM_E4M3) || lddy < hidden || lds < hidden || lddx < hidden ||
        (dsum && lddsum < hidden))
        return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && hidden > 0 && (!dy || !s || !weight || !rstd || !dx)) return GEMM_ERR_INVALID_ARG;
    if (st != GEMM_OK) return st;
    if (misaligned(dy, 2) || misaligned(s, 2) || misaligned(weight, 2) || misaligned(rstd, 4) || misaligned(dsum, 2) ||
        misaligned(dx, 2) || misaligned(dweight, 4))
        return GEMM_ERR_UNSUPPORTED;
    if (hidden == 0) return GEMM_OK;
    if (rows == 0) {
        if (!dweight) return GEMM_OK;
        return cudaMemsetAsync(dweight, 0, (size_t)hidden * sizeof(float), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? GEMM_OK
                   : GEMM_ERR_CUDA;
    }
    if (dweight && (!workspace || misaligned(workspace, 16))) return GEMM_ERR_WORKSPACE;
    NormGradArgs a{};
    a.dy = static_cast<const uint16_t*>(dy);
    a.s = static_cast<const uint16_t*>(s);
    a.weight = static_cast<const uint16_t*>(weight);
    a.dsum = static_cast<const uint16_t*>(dsum);
    a.rstd = rstd;
    a.lddy = lddy;
    a.lds = lds;
    a.lddsum = dsum ? lddsum : 0;
    a.rows = rows;
    a.lddx = lddx;
    a.hidden = (int)hidden;
    a.dx = static_cast<uint16_t*>(dx);
    a.part = dweight ? static_cast<float*>(workspace) : nullptr;
    const bool al = whole_chunks(hidden, {dy, s, weight, dsum, dx}, {lddy, lds, a.lddsum, lddx}, {}, {});
    return (dtype == GEMM_BF16 ? norm_grad<__nv_bfloat16> : norm_grad<__half>)(a, al, dweight, stream);
}

}  // extern "C"
