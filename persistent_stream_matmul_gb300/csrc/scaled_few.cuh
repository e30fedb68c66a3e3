// Scaled products of a few rows of A (one generated token, a small batch) and other
// small ones, both operands with the summed dimension contiguous.
//
// Bound by the reading of B: 2 M operations a byte of it.  What a small product
// pays beside that is latency, so this kernel has no ring, no tensor memory and
// no second pass: a warp reads its rows of B from global memory straight into the
// fragments of m16n8k32 products, whose rows are B's and whose columns are the rows
// of A.  A sum does not depend on the order of k, so a thread takes 32 neighbouring
// bytes of a row (four threads a 128-byte group) and gives four of them at a time
// to a product, where the fragment's layout has k 4t .. 4t + 3 and 16 + 4t .. ;
// A's fragments are read the same way.
//
// The k-blocks are cut into one part a warp of the block; the parts are added in
// ascending k through shared memory.
#pragma once
#include "scaled_kernel.cuh"

namespace psm {

constexpr int F_WARPS = 8;
// k-blocks of a warp in flight (one for more than 16 rows), and blocks an SM.  Bytes in
// flight against registers: us for one row, 14336 x 4096 / 4096 x 14336 / 4096 x 4096, with 2
// and 2 blocks 15.0 / 14.6 / 5.9; 2 and 3 15.3 / 20.8 / 7.7; 1 and 3 13.1 / 17.2 / 6.3; 3 and 2
// 15.5 / 14.0 / 6.2 (16 rows 18.5, 32.4, 24.9 and 30.1); with 32 rows of B a warp 17.2 / 19.7 /
// 8.2.  24 rows of 4096 x 4096, 1 and 2 8.4, 2 and 1 10.7.
constexpr int F_BLOCKS = 2, F_RESIDENT = 2;
constexpr int F_MOST_ROWS = 32;  // of A, a block

// k-blocks of a warp that are brought into L2 ahead.  us in a chain of products of one row,
// with 0, 2, 8: 14336 x 4096 15.0 / 14.3 / 14.5, 4096 x 14336 14.7 / 14.2 / 15.1, 4096 x 4096
// 5.9 / 5.1 / 5.0.
constexpr int F_PREFETCH = 2;

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

struct FewParams {
    const uint8_t *a, *b;
    ScaledScales sa, sb;
    void* out;
    int64_t K, N;
    int32_t M, kb, out_dtype;
};

template <bool A_E5M2, bool B_E5M2>
__device__ __forceinline__ void mma_f8_m16n8k32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
#define PSM_MMA_F8(TA, TB)                                                                          \
    asm("mma.sync.aligned.m16n8k32.row.col.f32." TA "." TB ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, " \
        "{%8, %9}, {%0, %1, %2, %3};"                                                               \
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                            \
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]))
    if constexpr (A_E5M2 && B_E5M2) PSM_MMA_F8("e5m2", "e5m2");
    else if constexpr (A_E5M2) PSM_MMA_F8("e5m2", "e4m3");
    else if constexpr (B_E5M2) PSM_MMA_F8("e4m3", "e5m2");
    else PSM_MMA_F8("e4m3", "e4m3");
#undef PSM_MMA_F8
}

// 32 bytes; rows start at 16-byte boundaries, and end at one (`bytes` of them are there).
__device__ __forceinline__ void few_load(const uint8_t* p, int64_t bytes, uint32_t (&w)[8]) {
    uint4 x{}, y{};
    if (bytes > 0) x = *reinterpret_cast<const uint4*>(p);
    if (bytes > 16) y = *reinterpret_cast<const uint4*>(p + 16);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
}

// NT: tiles of 8 rows of A.
template <bool W_E5M2, bool X_E5M2, int NT>
__global__ void __launch_bounds__(32 * F_WARPS, F_RESIDENT) few_kernel(const __grid_constant__ FewParams p) {
    constexpr int U = NT <= 2 ? F_BLOCKS : 1;
    __shared__ float part[F_WARPS][16][NT * 8 + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int m0 = blockIdx.y * (NT * 8), rows = min(p.M - m0, NT * 8);  // of A
    // rows past the end read the last one's
    const uint8_t* b[2];
    const float* sb[2];
    const uint8_t* a[NT];
    const float* sa[NT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t n = min(n0 + h * 8 + g, p.N - 1);
        b[h] = p.b + n * p.K + t * 32;
        sb[h] = p.sb.s + (n >> p.sb.shift) * p.sb.row;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        a[j] = p.a + (int64_t)(m0 + min(j * 8 + g, rows - 1)) * p.K + t * 32;
#pragma unroll
        for (int h = 0; h < 2; ++h) sa[j][h] = p.sa.s + (int64_t)((m0 + min(j * 8 + t * 2 + h, rows - 1)) >> p.sa.shift) * p.sa.row;
    }
    const int k0 = (int)((int64_t)p.kb * warp / F_WARPS), k1 = (int)((int64_t)p.kb * (warp + 1) / F_WARPS);
    float acc[NT][4] = {};
    // While the kernel before drains, this warp's lines of B are brought into L2 (and
    // no further: what that kernel may still write there is not read before the wait).
#pragma unroll 1
    for (int kb = k0 + (lane >> 4); kb < min(k1, k0 + F_PREFETCH); kb += 2)
        prefetch_l2(p.b + min(n0 + (lane & 15), p.N - 1) * p.K + (int64_t)kb * S_BK);
    grid_dependency_wait();
    grid_launch_dependents();
#pragma unroll 1
    for (int kb0 = k0; kb0 < k1; kb0 += U) {
        uint32_t wb[U][2][8], wa[U][NT][8];
        float fb[U][2], fa[U][NT][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = kb0 + u;
            // nothing is read past this warp's part (or the row)
            const int64_t at = (int64_t)kb * S_BK, left = kb < k1 ? p.K - at - t * 32 : 0;
            const int64_t gb = (int64_t)min(kb, k1 - 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) few_load(b[h] + at, left, wb[u][h]);
#pragma unroll
            for (int j = 0; j < NT; ++j) few_load(a[j] + at, left, wa[u][j]);
#pragma unroll
            for (int h = 0; h < 2; ++h) fb[u][h] = sb[h][gb * p.sb.group];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) fa[u][j][h] = sa[j][h][gb * p.sa.group];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (kb0 + u >= k1) break;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float d[4] = {};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t x[4] = {wb[u][0][2 * s], wb[u][1][2 * s], wb[u][0][2 * s + 1], wb[u][1][2 * s + 1]};
                    const uint32_t y[2] = {wa[u][j][2 * s], wa[u][j][2 * s + 1]};
                    mma_f8_m16n8k32<W_E5M2, X_E5M2>(d, x, y);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[j][c] = fmaf(d[c], fb[u][c >> 1] * fa[u][j][c & 1], acc[j][c]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) part[warp][(c >> 1) * 8 + g][j * 8 + t * 2 + (c & 1)] = acc[j][c];
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * rows; e += 32 * F_WARPS) {
        const int r = e % (16), m = e / (16);
        if (n0 + r >= p.N) continue;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < F_WARPS; ++w) sum += part[w][r][m];
        scaled_store(p.out, p.out_dtype, (int64_t)(m0 + m) * p.N + n0 + r, sum);
    }
}

}  // namespace psm
