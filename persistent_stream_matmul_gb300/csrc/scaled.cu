// Scaled products of include/gemm_scaled.h: plans, launches and the C entry
// points.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <new>

#include "gemm_scaled.h"
#include "ptx.cuh"
#include "rows.cuh"

using namespace psm;

struct gemm_scaled_plan {
    int64_t M, N, K;
    int type_a, type_b, out_dtype, layout_a, layout_b, scale_a, scale_b, device;
};

namespace {

constexpr int GROUP = GEMM_SCALE_GROUP;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

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

// One operand: element (r, k) at q[r * row + k * col], its scale at
// s[(r >> shift) * s_row + (k / 128) * s_group].
struct Operand {
    const uint8_t* q;
    const float* s;
    int64_t row, col, s_row, s_group, rows;
    int shift, e5m2;
};

__device__ __forceinline__ float value(uint8_t v, int e5m2) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, e5m2 ? __NV_E5M2 : __NV_E4M3)));
}

// 64 x 64 of C a block, 4 x 4 a thread; a group's sum is scaled and added to the
// sums before it.
__global__ void __launch_bounds__(256) scaled_kernel(Operand a, Operand b, int64_t K, void* c, int out_dtype) {
    __shared__ float as[32][65], bs[32][65];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * 64, n0 = (int64_t)blockIdx.y * 64;
    grid_dependency_wait();
    float acc[4][4] = {};
    for (int64_t g = 0; g * GROUP < K; ++g) {
        float part[4][4] = {};
        for (int64_t k0 = g * GROUP; k0 < g * GROUP + GROUP; k0 += 32) {
            __syncthreads();
            for (int i = threadIdx.x; i < 64 * 32; i += 256) {
                const int r = i >> 5, k = i & 31;
                as[k][r] = m0 + r < a.rows && k0 + k < K ? value(a.q[(m0 + r) * a.row + (k0 + k) * a.col], a.e5m2) : 0.f;
                bs[k][r] = n0 + r < b.rows && k0 + k < K ? value(b.q[(n0 + r) * b.row + (k0 + k) * b.col], b.e5m2) : 0.f;
            }
            __syncthreads();
            for (int k = 0; k < 32; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) part[i][j] = fmaf(as[k][ty * 4 + i], bs[k][tx * 4 + j], part[i][j]);
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
                if (m < a.rows && n < b.rows)
                    acc[i][j] = fmaf(part[i][j], a.s[(m >> a.shift) * a.s_row + g * a.s_group] * b.s[(n >> b.shift) * b.s_row + g * b.s_group], acc[i][j]);
            }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j, at = m * b.rows + n;
            if (m >= a.rows || n >= b.rows) continue;
            if (out_dtype == GEMM_F32) static_cast<float*>(c)[at] = acc[i][j];
            else if (out_dtype == GEMM_BF16) static_cast<__nv_bfloat16*>(c)[at] = __float2bfloat16_rn(acc[i][j]);
            else static_cast<__half*>(c)[at] = __float2half_rn(acc[i][j]);
        }
}

// k_major: the summed dimension is contiguous.
Operand operand(const void* q, const float* s, int64_t rows, int64_t K, bool k_major, int scale, int type) {
    Operand o{};
    o.q = static_cast<const uint8_t*>(q);
    o.s = s;
    o.rows = rows;
    o.row = k_major ? K : 1;
    o.col = k_major ? 1 : rows;
    o.e5m2 = type == GEMM_E5M2;
    if (scale == GEMM_SCALE_VECTOR) {
        o.s_row = 1;
        o.s_group = rows;
    } else {
        o.shift = 7;
        o.s_row = k_major ? cdiv(K, GROUP) : 1;
        o.s_group = k_major ? 1 : cdiv(rows, GROUP);
    }
    return o;
}

bool bad(int v) { return v != 0 && v != 1; }

}  // namespace

extern "C" {

gemm_status_t gemm_scaled_plan_create(gemm_scaled_plan_t* out, int64_t M, int64_t N, int64_t K,
                                      gemm_fp8_t type_a, gemm_fp8_t type_b, int out_dtype,
                                      gemm_layout_t layout_a, gemm_layout_t layout_b,
                                      gemm_scale_t scale_a, gemm_scale_t scale_b) {
    if (!out || M < 0 || N < 0 || K < 0 || bad(type_a) || bad(type_b) || bad(layout_a) || bad(layout_b) || bad(scale_a) ||
        bad(scale_b) || (out_dtype != GEMM_F16 && out_dtype != GEMM_BF16 && out_dtype != GEMM_F32))
        return GEMM_ERR_INVALID_ARG;
    if (M > MAX_INDEX || N > MAX_INDEX || K > MAX_INDEX || (layout_a == GEMM_ROW_MAJOR ? K : M) % 16 ||
        (layout_b == GEMM_COL_MAJOR ? K : N) % 16 || cdiv(N, 64) > 65535)
        return GEMM_ERR_UNSUPPORTED;
    int count = 0, dev = 0, major = 0, minor = 0;
    if (cudaGetDeviceCount(&count) != cudaSuccess || count == 0) {
        cudaGetLastError();
        return GEMM_ERR_NO_DEVICE;
    }
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return GEMM_ERR_CUDA;
    if (major != 10 || minor != 3) return GEMM_ERR_NO_DEVICE;
    gemm_scaled_plan* p = new (std::nothrow) gemm_scaled_plan{M, N, K, type_a, type_b, out_dtype, layout_a, layout_b, scale_a, scale_b, dev};
    if (!p) return GEMM_ERR_CUDA;
    *out = p;
    return GEMM_OK;
}

gemm_status_t gemm_scaled_workspace_size(gemm_scaled_plan_t p, size_t* bytes) {
    if (!p || !bytes) return GEMM_ERR_INVALID_ARG;
    *bytes = 0;
    return GEMM_OK;
}

gemm_status_t gemm_scaled_run(gemm_scaled_plan_t p, const void* A, const float* scales_a,
                              const void* B, const float* scales_b, void* C, void* workspace,
                              gemm_stream_t stream) {
    if (!p) return GEMM_ERR_INVALID_ARG;
    if (p->M == 0 || p->N == 0) return GEMM_OK;
    if (!C || (p->K > 0 && (!A || !B || !scales_a || !scales_b))) return GEMM_ERR_INVALID_ARG;
    const size_t size = p->out_dtype == GEMM_F32 ? 4 : 2;
    if (misaligned(A, 16) || misaligned(B, 16) || misaligned(C, size) || misaligned(scales_a, 4) || misaligned(scales_b, 4))
        return GEMM_ERR_UNSUPPORTED;
    DeviceGuard guard(p->device);
    if (!guard.ok) return GEMM_ERR_CUDA;
    const Operand a = operand(A, scales_a, p->M, p->K, p->layout_a == GEMM_ROW_MAJOR, p->scale_a, p->type_a);
    const Operand b = operand(B, scales_b, p->N, p->K, p->layout_b == GEMM_COL_MAJOR, p->scale_b, p->type_b);
    return launch(scaled_kernel, dim3((unsigned)cdiv(p->M, 64), (unsigned)cdiv(p->N, 64)), dim3(256), 0, stream, a, b, p->K, C, p->out_dtype);
}

gemm_status_t gemm_scaled_last_status(gemm_scaled_plan_t p, gemm_stream_t stream) {
    if (!p) return GEMM_ERR_INVALID_ARG;
    DeviceGuard guard(p->device);
    if (!guard.ok) return GEMM_ERR_CUDA;
    return cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status_t gemm_scaled_plan_destroy(gemm_scaled_plan_t p) {
    delete p;
    return GEMM_OK;
}

}  // extern "C"
