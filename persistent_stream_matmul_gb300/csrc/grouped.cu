// Grouped products of include/gemm_moe.h: plans, launches and the C entry points.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <new>

#include "gemm_moe.h"
#include "ptx.cuh"

using namespace psm;

namespace {

constexpr int64_t MAX_INDEX = (1ll << 31) - 1024;

__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// Offset g made monotone and in range: the largest of offsets[0 .. g], within [0, rows].
__device__ int bounded_offset(const int32_t* offsets, int g, int rows) {
    int v = 0;
    for (int i = 0; i <= g; ++i) v = max(v, offsets[i]);
    return min(v, rows);
}

constexpr int TILE = 64, KT = 16;

// One 64 x 64 tile of out = P^T-like products at a time, 256 threads of 4 x 4
// outputs.  pe(i, k) and qe(j, k) give the operands' elements, st(i, j, v) stores.
template <typename PE, typename QE, typename ST>
__device__ void tile_product(float (*sp)[TILE], float (*sq)[TILE], int64_t klen, PE pe, QE qe, ST st) {
    float acc[4][4] = {};
    const int ti = (threadIdx.x / 16) * 4, tj = (threadIdx.x % 16) * 4;
    for (int64_t k0 = 0; k0 < klen; k0 += KT) {
        __syncthreads();
        for (int x = threadIdx.x; x < TILE * KT; x += 256) {
            const int i = x % TILE, k = x / TILE;
            sp[k][i] = k0 + k < klen ? pe(i, k0 + k) : 0.f;
            sq[k][i] = k0 + k < klen ? qe(i, k0 + k) : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < KT; ++k)
            for (int a = 0; a < 4; ++a)
                for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(sp[k][ti + a], sq[k][tj + b], acc[a][b]);
    }
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) st(ti + a, tj + b, acc[a][b]);
}

template <typename T>
__global__ void __launch_bounds__(256)
    rows_kernel(const T* A, const T* B, T* C, const int32_t* offsets, int groups, int rows, int N, int K,
                bool b_col) {
    __shared__ float sp[KT][TILE], sq[KT][TILE];
    grid_dependency_wait();
    grid_launch_dependents();
    const int g = blockIdx.y, n0 = blockIdx.x * TILE;
    const int r_begin = bounded_offset(offsets, g, rows);
    const bool tail = g == groups;  // the unused rows
    const int r_end = tail ? rows : bounded_offset(offsets, g + 1, rows);
    const T* Bg = B + (int64_t)g * N * K;
    for (int64_t r0 = r_begin; r0 < r_end; r0 += TILE)
        tile_product(
            sp, sq, tail ? 0 : K,
            [&](int i, int64_t k) { return r0 + i < r_end ? to_f(A[(r0 + i) * K + k]) : 0.f; },
            [&](int j, int64_t k) {
                return n0 + j < N ? to_f(b_col ? Bg[(int64_t)(n0 + j) * K + k] : Bg[k * N + n0 + j]) : 0.f;
            },
            [&](int i, int j, float v) {
                if (r0 + i < r_end && n0 + j < N) C[(r0 + i) * N + n0 + j] = from_f<T>(v);
            });
}

template <typename T>
__global__ void __launch_bounds__(256)
    inner_kernel(const T* A, const T* B, T* C, const int32_t* offsets, int groups, int rows, int N, int K,
                 bool c_col) {
    __shared__ float sp[KT][TILE], sq[KT][TILE];
    grid_dependency_wait();
    grid_launch_dependents();
    const int n0 = blockIdx.x * TILE, k0 = blockIdx.y * TILE, g = blockIdx.z;
    const int64_t r0 = bounded_offset(offsets, g, rows), r1 = bounded_offset(offsets, g + 1, rows);
    T* Cg = C + (int64_t)g * N * K;
    tile_product(
        sp, sq, r1 - r0, [&](int i, int64_t r) { return k0 + i < K ? to_f(A[(r0 + r) * K + k0 + i]) : 0.f; },
        [&](int j, int64_t r) { return n0 + j < N ? to_f(B[(r0 + r) * N + n0 + j]) : 0.f; },
        [&](int i, int j, float v) {
            if (k0 + i < K && n0 + j < N)
                Cg[c_col ? (int64_t)(n0 + j) * K + k0 + i : (int64_t)(k0 + i) * N + n0 + j] = from_f<T>(v);
        });
}

struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) { ok = false; return; }
        if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

}  // namespace

struct gemm_grouped_plan {
    int64_t groups, rows, N, K;
    int kind, dtype, layout_b, device, num_sms;
    int* d_status;
};

extern "C" {

gemm_status_t gemm_grouped_plan_create(gemm_grouped_plan_t* out, gemm_grouped_kind_t kind,
                                       int64_t groups, int64_t rows, int64_t N, int64_t K,
                                       gemm_dtype_t dtype, gemm_layout_t layout_b) {
    if (!out || groups < 1 || rows < 0 || N < 0 || K < 0 ||
        (kind != GEMM_GROUPED_ROWS && kind != GEMM_GROUPED_INNER) ||
        (dtype != GEMM_F16 && dtype != GEMM_BF16) ||
        (layout_b != GEMM_ROW_MAJOR && layout_b != GEMM_COL_MAJOR))
        return GEMM_ERR_INVALID_ARG;
    if (groups > GEMM_MOE_MAX_EXPERTS || rows > MAX_INDEX || N > MAX_INDEX || K > MAX_INDEX || N % 8 || K % 8)
        return GEMM_ERR_UNSUPPORTED;
    int dev = 0, count = 0, major = 0, minor = 0, sms = 0;
    if (cudaGetDeviceCount(&count) != cudaSuccess || count == 0) {
        cudaGetLastError();
        return GEMM_ERR_NO_DEVICE;
    }
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return GEMM_ERR_CUDA;
    if (major != 10 || minor != 3) return GEMM_ERR_NO_DEVICE;
    gemm_grouped_plan* p = new (std::nothrow) gemm_grouped_plan();
    if (!p) return GEMM_ERR_CUDA;
    p->groups = groups;
    p->rows = rows;
    p->N = N;
    p->K = K;
    p->kind = kind;
    p->dtype = dtype;
    p->layout_b = layout_b;
    p->device = dev;
    p->num_sms = sms;
    if (cudaMalloc(&p->d_status, sizeof(int)) != cudaSuccess ||
        cudaMemset(p->d_status, 0, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        if (p->d_status) cudaFree(p->d_status);
        delete p;
        return GEMM_ERR_CUDA;
    }
    *out = p;
    return GEMM_OK;
}

gemm_status_t gemm_grouped_workspace_size(gemm_grouped_plan_t p, size_t* bytes) {
    if (!p || !bytes) return GEMM_ERR_INVALID_ARG;
    *bytes = 0;
    return GEMM_OK;
}

gemm_status_t gemm_grouped_run(gemm_grouped_plan_t p, const void* A, const void* B, void* C,
                               const int32_t* offsets, void* workspace, gemm_stream_t stream) {
    if (!p) return GEMM_ERR_INVALID_ARG;
    const bool inner = p->kind == GEMM_GROUPED_INNER;
    if (p->N == 0 || (inner ? p->K : p->rows) == 0) return GEMM_OK;  // C is empty
    const bool sums = inner ? p->rows > 0 : p->K > 0;                // something to sum
    if (!C || !offsets || (sums && (!A || !B))) return GEMM_ERR_INVALID_ARG;
    if (((uintptr_t)A & 15u) || ((uintptr_t)B & 15u) || ((uintptr_t)C & 15u) || ((uintptr_t)offsets & 3u))
        return GEMM_ERR_UNSUPPORTED;
    (void)workspace;
    DeviceGuard guard(p->device);
    if (!guard.ok) return GEMM_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!sums) {
        const size_t bytes = 2 * (size_t)p->N * (size_t)(inner ? p->groups * p->K : p->rows);
        return cudaMemsetAsync(C, 0, bytes, st) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
    }
    const unsigned nt = (unsigned)((p->N + TILE - 1) / TILE), kt = (unsigned)((p->K + TILE - 1) / TILE);
    const bool col = p->layout_b == GEMM_COL_MAJOR, bf = p->dtype == GEMM_BF16;
    const int G = (int)p->groups, R = (int)p->rows, N = (int)p->N, K = (int)p->K;
    using BF = __nv_bfloat16;
    using HF = __half;
    if (inner) {
        const dim3 grid(nt, kt, G);
        if (bf) inner_kernel<BF><<<grid, 256, 0, st>>>((const BF*)A, (const BF*)B, (BF*)C, offsets, G, R, N, K, col);
        else inner_kernel<HF><<<grid, 256, 0, st>>>((const HF*)A, (const HF*)B, (HF*)C, offsets, G, R, N, K, col);
    } else {
        const dim3 grid(nt, G + 1, 1);
        if (bf) rows_kernel<BF><<<grid, 256, 0, st>>>((const BF*)A, (const BF*)B, (BF*)C, offsets, G, R, N, K, col);
        else rows_kernel<HF><<<grid, 256, 0, st>>>((const HF*)A, (const HF*)B, (HF*)C, offsets, G, R, N, K, col);
    }
    if (cudaGetLastError() != cudaSuccess) return GEMM_ERR_LAUNCH;
    return GEMM_OK;
}

gemm_status_t gemm_grouped_last_status(gemm_grouped_plan_t p, gemm_stream_t stream) {
    if (!p) return GEMM_ERR_INVALID_ARG;
    DeviceGuard guard(p->device);
    if (!guard.ok) return GEMM_ERR_CUDA;
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return GEMM_ERR_CUDA;
    int h = 0;
    if (cudaMemcpy(&h, p->d_status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return GEMM_ERR_CUDA;
    if (h == 0) return GEMM_OK;
    return cudaMemset(p->d_status, 0, sizeof(int)) == cudaSuccess ? GEMM_ERR_TIMEOUT : GEMM_ERR_CUDA;
}

gemm_status_t gemm_grouped_plan_destroy(gemm_grouped_plan_t p) {
    if (!p) return GEMM_OK;
    if (p->d_status) cudaFree(p->d_status);
    delete p;
    return GEMM_OK;
}

}  // extern "C"
