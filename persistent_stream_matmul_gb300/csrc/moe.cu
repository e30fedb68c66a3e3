// Mixture-of-experts row operators of include/gemm_moe.h: the stable sort of
// the slots by expert, and the row movements with their gradients.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

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

// Exclusive prefix of v over the block and its total, through ballots (v is
// 0 or 1).  `warps` holds one count per warp.
__device__ __forceinline__ int block_rank(bool v, int* warps, int& total) {
    const unsigned m = __ballot_sync(0xffffffffu, v);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    __syncthreads();
    if (lane == 0) warps[warp] = __popc(m);
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp) before += warps[w];
        total += warps[w];
    }
    return before + __popc(m & ((1u << lane) - 1));
}

// Block e ranks the slots of expert e; block `experts` handles the dropped
// ones.  Every block reads all ids: E * S reads.
template <typename I>
__global__ void __launch_bounds__(512)
    sort_kernel(const I* ids, int64_t ld, int64_t total, int topk, int experts, int32_t* offsets,
                int32_t* rows, int32_t* slots) {
    __shared__ int warps[16];
    grid_dependency_wait();
    grid_launch_dependents();
    const int e = blockIdx.x;
    auto key = [&](int64_t s) {
        const I v = ids[(s / topk) * ld + s % topk];
        return v >= 0 && v < experts ? (int)v : experts;
    };
    int first = 0;
    for (int64_t b = 0; b < total; b += blockDim.x) {
        const int64_t s = b + threadIdx.x;
        int n;
        block_rank(s < total && key(s) < e, warps, n);
        first += n;
    }
    if (threadIdx.x == 0) offsets[e] = first;
    int at = first;
    for (int64_t b = 0; b < total; b += blockDim.x) {
        const int64_t s = b + threadIdx.x;
        const bool mine = s < total && key(s) == e;
        int n;
        const int r = at + block_rank(mine, warps, n);
        if (mine) {
            rows[s] = e < experts ? r : -1;
            if (e < experts) slots[r] = (int32_t)s;
        }
        at += n;
    }
    if (e == experts)
        for (int64_t r = first + threadIdx.x; r < total; r += blockDim.x) slots[r] = -1;
}

// One block per token: out[rows[t, j]] = w * x[t].  GRAD also writes dweights.
template <typename T, bool GRAD>
__global__ void __launch_bounds__(256)
    spread_kernel(const T* x, int64_t ldx, const T* ys, int64_t ldys, const int32_t* rows,
                  const int32_t* slots, const float* weights, int topk, int64_t total, int hidden,
                  T* out, int64_t ldo, float* dweights) {
    __shared__ float part[8];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t t = blockIdx.x;
    for (int j = 0; j < topk; ++j) {
        const int64_t s = t * topk + j, r = rows[s];
        const bool kept = r >= 0 && r < total;
        float dot = 0.f;
        if (kept) {
            const float w = GRAD ? weights[s] : 1.f;
            for (int h = threadIdx.x; h < hidden; h += blockDim.x) {
                const T v = x[t * ldx + h];
                out[r * ldo + h] = GRAD ? from_f<T>(w * to_f(v)) : v;
                if (GRAD) dot = fmaf(to_f(v), to_f(ys[r * ldys + h]), dot);
            }
        }
        if (GRAD) {
            for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            __syncthreads();
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
            __syncthreads();
            if (threadIdx.x == 0) {
                float sum = 0.f;
                for (int i = 0; i < (int)blockDim.x / 32; ++i) sum += part[i];
                dweights[s] = sum;
            }
        }
        if (slots[s] < 0)  // row s is unused
            for (int h = threadIdx.x; h < hidden; h += blockDim.x) out[s * ldo + h] = from_f<T>(0.f);
    }
}

// One block per token: out[t] = the sum over j of w[t, j] * src[rows[t, j]].
template <typename T, bool WEIGHTED>
__global__ void __launch_bounds__(256)
    gather_kernel(const T* src, int64_t lds, const int32_t* rows, const float* weights, int topk,
                  int64_t total, int hidden, T* out, int64_t ldo) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t t = blockIdx.x;
    for (int h = threadIdx.x; h < hidden; h += blockDim.x) {
        float acc = 0.f;
        for (int j = 0; j < topk; ++j) {
            const int64_t r = rows[t * topk + j];
            if (r < 0 || r >= total) continue;
            const float v = to_f(src[r * lds + h]);
            acc = WEIGHTED ? fmaf(weights[t * topk + j], v, acc) : acc + v;
        }
        out[t * ldo + h] = from_f<T>(acc);
    }
}

template <typename... P, typename... A>
gemm_status_t launch(void (*kernel)(P...), int64_t grid, int block, gemm_stream_t stream, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)block, 1, 1);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    // as the products: the grid may start while the kernel before it drains,
    // and waits for it before it touches global memory
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

bool misaligned(const void* p, size_t size) { return ((uintptr_t)p & (size - 1)) != 0; }

// The checks that the row operators share; `ok` false when there is nothing to do.
gemm_status_t check_rows(int64_t tokens, int64_t topk, int64_t hidden, int dtype) {
    if (tokens < 0 || topk < 1 || hidden < 0 || (dtype != GEMM_F16 && dtype != GEMM_BF16))
        return GEMM_ERR_INVALID_ARG;
    if (topk > MAX_INDEX || tokens > MAX_INDEX / topk || hidden > MAX_INDEX) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

template <typename T>
gemm_status_t gather(const void* src, int64_t lds, const int32_t* rows, const float* weights,
                     int64_t tokens, int64_t topk, int64_t hidden, void* out, int64_t ldo,
                     gemm_stream_t stream) {
    return launch(weights ? gather_kernel<T, true> : gather_kernel<T, false>, tokens, 256, stream,
                  static_cast<const T*>(src), lds, rows, weights, (int)topk, tokens * topk, (int)hidden,
                  static_cast<T*>(out), ldo);
}

template <typename T>
gemm_status_t spread(const void* x, int64_t ldx, const void* ys, int64_t ldys, const int32_t* rows,
                     const int32_t* slots, const float* weights, int64_t tokens, int64_t topk,
                     int64_t hidden, void* out, int64_t ldo, float* dweights, gemm_stream_t stream) {
    return launch(weights ? spread_kernel<T, true> : spread_kernel<T, false>, tokens, 256, stream,
                  static_cast<const T*>(x), ldx, static_cast<const T*>(ys), ldys, rows, slots, weights,
                  (int)topk, tokens * topk, (int)hidden, static_cast<T*>(out), ldo, dweights);
}

gemm_status_t check_sort(int64_t tokens, int64_t topk, int64_t experts) {
    if (tokens < 0 || topk < 1 || experts < 1) return GEMM_ERR_INVALID_ARG;
    if (experts > GEMM_MOE_MAX_EXPERTS || topk > MAX_INDEX || tokens > MAX_INDEX / topk)
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t gemm_moe_sort_workspace_size(int64_t tokens, int64_t topk, int64_t experts,
                                           size_t* bytes) {
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = check_sort(tokens, topk, experts);
    if (st == GEMM_OK) *bytes = 0;
    return st;
}

gemm_status_t gemm_moe_sort(const void* ids, gemm_index_t id_type, int64_t ld_ids, int64_t tokens,
                            int64_t topk, int64_t experts, int32_t* offsets, int32_t* rows,
                            int32_t* slots, void* workspace, gemm_stream_t stream) {
    const gemm_status_t st = check_sort(tokens, topk, experts);
    if (st == GEMM_ERR_INVALID_ARG || (id_type != GEMM_INDEX_I32 && id_type != GEMM_INDEX_I64) ||
        ld_ids < topk || !offsets || (tokens > 0 && (!ids || !rows || !slots)))
        return GEMM_ERR_INVALID_ARG;
    if (st != GEMM_OK) return st;
    if (misaligned(ids, id_type == GEMM_INDEX_I64 ? 8 : 4) || misaligned(offsets, 4) ||
        misaligned(rows, 4) || misaligned(slots, 4))
        return GEMM_ERR_UNSUPPORTED;
    (void)workspace;
    if (id_type == GEMM_INDEX_I64)
        return launch(sort_kernel<int64_t>, experts + 1, 512, stream, static_cast<const int64_t*>(ids),
                      ld_ids, tokens * topk, (int)topk, (int)experts, offsets, rows, slots);
    return launch(sort_kernel<int32_t>, experts + 1, 512, stream, static_cast<const int32_t*>(ids),
                  ld_ids, tokens * topk, (int)topk, (int)experts, offsets, rows, slots);
}

gemm_status_t gemm_moe_dispatch(const void* x, int64_t ldx, const int32_t* rows,
                                const int32_t* slots, int64_t tokens, int64_t topk, int64_t hidden,
                                gemm_dtype_t dtype, void* xs, int64_t ldxs, gemm_stream_t stream) {
    const gemm_status_t st = check_rows(tokens, topk, hidden, dtype);
    if (st == GEMM_ERR_INVALID_ARG || ldx < hidden || ldxs < hidden) return GEMM_ERR_INVALID_ARG;
    if (tokens > 0 && hidden > 0 && (!x || !rows || !slots || !xs)) return GEMM_ERR_INVALID_ARG;
    if (st != GEMM_OK) return st;
    if (misaligned(x, 2) || misaligned(xs, 2) || misaligned(rows, 4) || misaligned(slots, 4))
        return GEMM_ERR_UNSUPPORTED;
    if (tokens == 0 || hidden == 0) return GEMM_OK;
    return spread<__half>(x, ldx, nullptr, 0, rows, slots, nullptr, tokens, topk, hidden, xs, ldxs,
                          nullptr, stream);  // a copy: the type does not matter
}

gemm_status_t gemm_moe_dispatch_grad(const void* dxs, int64_t lddxs, const int32_t* rows,
                                     int64_t tokens, int64_t topk, int64_t hidden,
                                     gemm_dtype_t dtype, void* dx, int64_t lddx,
                                     gemm_stream_t stream) {
    const gemm_status_t st = check_rows(tokens, topk, hidden, dtype);
    if (st == GEMM_ERR_INVALID_ARG || lddxs < hidden || lddx < hidden) return GEMM_ERR_INVALID_ARG;
    if (tokens > 0 && hidden > 0 && (!dxs || !rows || !dx)) return GEMM_ERR_INVALID_ARG;
    if (st != GEMM_OK) return st;
    if (misaligned(dxs, 2) || misaligned(dx, 2) || misaligned(rows, 4)) return GEMM_ERR_UNSUPPORTED;
    if (tokens == 0 || hidden == 0) return GEMM_OK;
    return (dtype == GEMM_BF16 ? gather<__nv_bfloat16> : gather<__half>)(
        dxs, lddxs, rows, nullptr, tokens, topk, hidden, dx, lddx, stream);
}

gemm_status_t gemm_moe_combine(const void* ys, int64_t ldys, const int32_t* rows,
                               const float* weights, int64_t tokens, int64_t topk, int64_t hidden,
                               gemm_dtype_t dtype, void* y, int64_t ldy, gemm_stream_t stream) {
    const gemm_status_t st = check_rows(tokens, topk, hidden, dtype);
    if (st == GEMM_ERR_INVALID_ARG || ldys < hidden || ldy < hidden) return GEMM_ERR_INVALID_ARG;
    if (tokens > 0 && hidden > 0 && (!ys || !rows || !weights || !y)) return GEMM_ERR_INVALID_ARG;
    if (st != GEMM_OK) return st;
    if (misaligned(ys, 2) || misaligned(y, 2) || misaligned(rows, 4) || misaligned(weights, 4))
        return GEMM_ERR_UNSUPPORTED;
    if (tokens == 0 || hidden == 0) return GEMM_OK;
    return (dtype == GEMM_BF16 ? gather<__nv_bfloat16> : gather<__half>)(
        ys, ldys, rows, weights, tokens, topk, hidden, y, ldy, stream);
}

gemm_status_t gemm_moe_combine_grad(const void* dy, int64_t lddy, const void* ys, int64_t ldys,
                                    const int32_t* rows, const int32_t* slots,
                                    const float* weights, int64_t tokens, int64_t topk,
                                    int64_t hidden, gemm_dtype_t dtype, void* dys, int64_t lddys,
                                    float* dweights, gemm_stream_t stream) {
    const gemm_status_t st = check_rows(tokens, topk, hidden, dtype);
    if (st == GEMM_ERR_INVALID_ARG || lddy < hidden || ldys < hidden || lddys < hidden)
        return GEMM_ERR_INVALID_ARG;
    if (tokens > 0 && (!rows || !slots || !weights || !dweights || (hidden > 0 && (!dy || !ys || !dys))))
        return GEMM_ERR_INVALID_ARG;
    if (st != GEMM_OK) return st;
    if (misaligned(dy, 2) || misaligned(ys, 2) || misaligned(dys, 2) || misaligned(rows, 4) ||
        misaligned(slots, 4) || misaligned(weights, 4) || misaligned(dweights, 4))
        return GEMM_ERR_UNSUPPORTED;
    if (tokens == 0) return GEMM_OK;  // hidden == 0 still has its (zero) dweights
    return (dtype == GEMM_BF16 ? spread<__nv_bfloat16> : spread<__half>)(
        dy, lddy, ys, ldys, rows, slots, weights, tokens, topk, hidden, dys, lddys, dweights, stream);
}

}  // extern "C"
