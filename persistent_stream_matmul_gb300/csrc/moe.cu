// Mixture-of-experts row operators of include/gemm_moe.h: the stable sort of
// the slots by expert, and the row movements with their gradients.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>

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

// ---------------------------------------------------------------- sort
// Stable counting sort.  The slots are cut into one contiguous chunk a block
// and, within it, one a warp; the row of a slot is
//   (slots of smaller experts) + (its expert's slots in earlier blocks)
//   + (in earlier warps) + (earlier in its warp).
// More than one block: count_kernel writes every block's histogram, and each
// block of place_kernel sums the table itself, so there is no third launch
// and no block waits for another.  The counts are whole numbers, so the order
// of the atomics in shared memory changes nothing.
constexpr int SORT_CHUNK = 4096;   // slots a block, until there are SORT_BLOCKS
constexpr int SORT_BLOCKS = 128;

struct SortArgs {
    int64_t ld, total, chunk;   // chunk: slots a block, a multiple of 1024
    int topk, experts, blocks;
};

template <typename I>
__device__ __forceinline__ int key_of(const I* ids, const SortArgs& a, int64_t s) {
    const I v = a.ld == a.topk ? ids[s] : ids[(s / a.topk) * a.ld + s % a.topk];
    return v >= 0 && v < (I)a.experts ? (int)v : a.experts;
}

template <typename I>
__global__ void __launch_bounds__(1024) count_kernel(const I* ids, SortArgs a, uint32_t* table) {
    __shared__ uint32_t hist[GEMM_MOE_MAX_EXPERTS];
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) hist[e] = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * a.chunk, s1 = min(a.total, s0 + a.chunk);
#pragma unroll 4
    for (int64_t s = s0 + threadIdx.x; s < s1; s += blockDim.x) {
        const int e = key_of(ids, a, s);
        if (e < a.experts) atomicAdd(&hist[e], 1u);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x)
        table[(size_t)blockIdx.x * a.experts + e] = hist[e];
}

template <typename I>
__global__ void __launch_bounds__(1024)
    place_kernel(const I* ids, SortArgs a, const uint32_t* table, int32_t* offsets, int32_t* rows,
                 int32_t* slots) {
    extern __shared__ uint32_t mine[];  // [warp][expert]: counts, then the next row
    __shared__ uint32_t before[GEMM_MOE_MAX_EXPERTS], all[GEMM_MOE_MAX_EXPERTS], sums[33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int E = a.experts;
    uint32_t* own = mine + warp * E;
    for (int i = threadIdx.x; i < warps * E; i += blockDim.x) mine[i] = 0;
    for (int e = threadIdx.x; e < E; e += blockDim.x) before[e] = all[e] = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();
    const int64_t per = a.chunk / warps;
    const int64_t w0 = blockIdx.x * a.chunk + warp * per, w1 = min(a.total, w0 + per);
    // this block's counts by warp
    for (int64_t b = w0; b < w1; b += 32) {
        const int e = b + lane < w1 ? key_of(ids, a, b + lane) : E;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e < E && lane == __ffs(same) - 1) own[e] += __popc(same);
        __syncwarp();
    }
    // all blocks' counts, and those of the blocks before this one
    if (a.blocks > 1) {
        const int parts = max(1, (int)blockDim.x / E);
        for (int i = threadIdx.x; i < parts * E; i += blockDim.x) {
            const int e = i % E;
            uint32_t sum = 0, prior = 0;
#pragma unroll 4
            for (int b = i / E; b < a.blocks; b += parts) {
                const uint32_t c = table[(size_t)b * E + e];
                sum += c;
                prior += b < (int)blockIdx.x ? c : 0;
            }
            atomicAdd(&all[e], sum);
            atomicAdd(&before[e], prior);
        }
        __syncthreads();
    } else {
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += blockDim.x)
            for (int w = 0; w < warps; ++w) all[e] += mine[w * E + e];
        __syncthreads();
    }
    // exclusive sum over the experts, blockDim.x at a time
    uint32_t carry = 0;
    for (int b = 0; b < E; b += blockDim.x) {
        const int e = b + threadIdx.x;
        const uint32_t c = e < E ? all[e] : 0;
        uint32_t v = c;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        if (warp == 0) {
            uint32_t x = lane < warps ? sums[lane] : 0;
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += u;
            }
            sums[lane] = x;
        }
        __syncthreads();
        const uint32_t first = carry + v - c + (warp > 0 ? sums[warp - 1] : 0);
        carry += sums[warps - 1];
        if (e < E) {
            uint32_t at = first + before[e];
            for (int w = 0; w < warps; ++w) {
                const uint32_t n = mine[w * E + e];
                mine[w * E + e] = at;
                at += n;
            }
            if (blockIdx.x == 0) offsets[e] = (int32_t)first;
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = (int32_t)carry;
    for (int64_t b = w0; b < w1; b += 32) {
        const bool in = b + lane < w1;
        const int e = in ? key_of(ids, a, b + lane) : E;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const uint32_t at = e < E ? own[e] : 0;
        __syncwarp();
        if (e < E) {
            const uint32_t r = at + __popc(same & ((1u << lane) - 1));
            rows[b + lane] = (int32_t)r;
            slots[r] = (int32_t)(b + lane);
            if (lane == __ffs(same) - 1) own[e] = at + __popc(same);
        } else if (in) {
            rows[b + lane] = -1;
        }
        __syncwarp();
    }
    for (int64_t r = carry + blockIdx.x * (int64_t)blockDim.x + threadIdx.x; r < a.total;
         r += (int64_t)gridDim.x * blockDim.x)
        slots[r] = -1;
}

SortArgs sort_shape(int64_t tokens, int64_t topk, int64_t experts) {
    SortArgs a{};
    a.total = tokens * topk;
    a.topk = (int)topk;
    a.experts = (int)experts;
    const int64_t even = (a.total + SORT_BLOCKS - 1) / SORT_BLOCKS;
    a.chunk = even > SORT_CHUNK ? (even + 1023) / 1024 * 1024 : SORT_CHUNK;
    a.blocks = (int)((a.total + a.chunk - 1) / a.chunk);
    if (a.blocks < 1) a.blocks = 1;
    return a;
}

// ---------------------------------------------------------------- row movements
// Bound by memory: every row is read or written once, V elements (16 bytes
// where all rows are 16-byte aligned, else one element) a thread and access.
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
    T v[V];
};

// i / d for 0 <= i, 0 < d: 32-bit division, several times shorter, where it does
__device__ __forceinline__ int64_t quotient(int64_t i, int d) {
    return i >> 32 ? i / d : (int64_t)((uint32_t)i / (uint32_t)d);
}

__device__ __forceinline__ bool in_range(int64_t r, int64_t total) { return r >= 0 && r < total; }

// out[rows[t, j]] = x[t] for one (token, chunk) a thread: x is read once.
template <typename T, int V>
__global__ void __launch_bounds__(256)
    dispatch_kernel(const T* x, int64_t ldx, const int32_t* rows, const int32_t* slots, int topk,
                    int64_t tokens, int chunks, T* out, int64_t ldo) {
    using Vt = Vec<T, V>;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t total = tokens * topk, n = tokens * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t t = quotient(i, chunks), h = (i - t * chunks) * V;
        const Vt v = *reinterpret_cast<const Vt*>(x + t * ldx + h);
        for (int j = 0; j < topk; ++j) {
            const int64_t s = t * topk + j, r = rows[s];
            if (in_range(r, total)) *reinterpret_cast<Vt*>(out + r * ldo + h) = v;
            if (slots[s] < 0) {  // row s is unused
                Vt z;
#pragma unroll
                for (int k = 0; k < V; ++k) z.v[k] = from_f<T>(0.f);
                *reinterpret_cast<Vt*>(out + s * ldo + h) = z;
            }
        }
    }
}

// out[t] = the sum over j of w[t, j] * src[rows[t, j]], one (token, chunk) a
// thread, the loads of U choices in flight together.
template <typename T, int V, int U, bool WEIGHTED>
__global__ void __launch_bounds__(256)
    gather_kernel(const T* src, int64_t lds, const int32_t* rows, const float* weights, int topk,
                  int64_t tokens, int chunks, T* out, int64_t ldo) {
    using Vt = Vec<T, V>;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t total = tokens * topk, n = tokens * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t t = quotient(i, chunks), h = (i - t * chunks) * V;
        float acc[V] = {};
        for (int j0 = 0; j0 < topk; j0 += U) {
            Vt v[U];
            float w[U];
            bool use[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t s = t * topk + j0 + u;
                const int64_t r = j0 + u < topk ? rows[s] : -1;
                use[u] = in_range(r, total);
                if (use[u]) {
                    v[u] = *reinterpret_cast<const Vt*>(src + r * lds + h);
                    w[u] = WEIGHTED ? weights[s] : 1.f;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (use[u])
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        acc[k] = WEIGHTED ? fmaf(w[u], to_f(v[u].v[k]), acc[k]) : acc[k] + to_f(v[u].v[k]);
        }
        Vt o;
#pragma unroll
        for (int k = 0; k < V; ++k) o.v[k] = from_f<T>(acc[k]);
        *reinterpret_cast<Vt*>(out + t * ldo + h) = o;
    }
}

// One block a token: dys[rows[t, j]] = w[t, j] * dy[t], and dweights[t, j] =
// dy[t] . ys[rows[t, j]], U choices at a time (dy is read again from the cache
// for the next U).  A thread adds its chunks in ascending order, then the
// warps' sums are added in order: fixed whatever the timing.
template <typename T, int V, int U>
__global__ void __launch_bounds__(256)
    combine_grad_kernel(const T* dy, int64_t lddy, const T* ys, int64_t ldys, const int32_t* rows,
                        const int32_t* slots, const float* weights, int topk, int64_t tokens, int chunks,
                        T* dys, int64_t lddys, float* dweights) {
    using Vt = Vec<T, V>;
    __shared__ float part[U][8];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t total = tokens * topk, t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    for (int j0 = 0; j0 < topk; j0 += U) {
        int64_t r[U];
        float w[U], dot[U];
        bool zero[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t s = t * topk + j0 + u;
            const bool in = j0 + u < topk;
            r[u] = in ? rows[s] : -1;
            if (!in_range(r[u], total)) r[u] = -1;
            w[u] = r[u] >= 0 ? weights[s] : 0.f;
            zero[u] = in && slots[s] < 0;
            dot[u] = 0.f;
        }
        for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
            const int64_t h = (int64_t)c * V;
            const Vt d = *reinterpret_cast<const Vt*>(dy + t * lddy + h);
            Vt y[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r[u] >= 0) y[u] = *reinterpret_cast<const Vt*>(ys + r[u] * ldys + h);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r[u] >= 0) {
                    Vt o;
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const float x = to_f(d.v[k]);
                        o.v[k] = from_f<T>(w[u] * x);
                        dot[u] = fmaf(x, to_f(y[u].v[k]), dot[u]);
                    }
                    *reinterpret_cast<Vt*>(dys + r[u] * lddys + h) = o;
                }
                if (zero[u]) {  // row t * topk + j is unused
                    Vt z;
#pragma unroll
                    for (int k = 0; k < V; ++k) z.v[k] = from_f<T>(0.f);
                    *reinterpret_cast<Vt*>(dys + (t * topk + j0 + u) * lddys + h) = z;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            for (int o = 16; o; o >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], o);
        __syncthreads();
        if (lane == 0)
#pragma unroll
            for (int u = 0; u < U; ++u) part[u][warp] = dot[u];
        __syncthreads();
        if (threadIdx.x < U && j0 + (int)threadIdx.x < topk) {
            float sum = 0.f;
            for (int i = 0; i < warps; ++i) sum += part[threadIdx.x][i];
            dweights[t * topk + j0 + threadIdx.x] = sum;
        }
    }
}

template <typename... P, typename... A>
gemm_status_t launch(void (*kernel)(P...), int64_t grid, int block, size_t smem, gemm_stream_t stream,
                     A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.dynamicSmemBytes = smem;
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

// 16 bytes an access when the rows allow it: aligned starts, leading
// dimensions and length.
bool wide(int64_t hidden, std::initializer_list<const void*> bases, std::initializer_list<int64_t> lds) {
    int64_t bits = hidden * 2;
    for (const void* b : bases) bits |= (int64_t)(uintptr_t)b;
    for (int64_t ld : lds) bits |= ld * 2;
    return (bits & 15) == 0;
}

// Blocks of 256 threads for n independent items; beyond 2^20 blocks the kernels
// stride over the rest.
int64_t blocks_for(int64_t n) { return std::min<int64_t>((n + 255) / 256, 1 << 20); }

template <typename T, int V>
gemm_status_t gather_v(const void* src, int64_t lds, const int32_t* rows, const float* weights,
                       int64_t tokens, int64_t topk, int64_t hidden, void* out, int64_t ldo,
                       gemm_stream_t stream) {
    const int chunks = (int)(hidden / V);
    auto* fn = weights ? (topk <= 2 ? gather_kernel<T, V, 2, true> : topk <= 4 ? gather_kernel<T, V, 4, true> : gather_kernel<T, V, 8, true>)
                       : (topk <= 2 ? gather_kernel<T, V, 2, false> : topk <= 4 ? gather_kernel<T, V, 4, false> : gather_kernel<T, V, 8, false>);
    return launch(fn, blocks_for(tokens * chunks), 256, 0, stream, static_cast<const T*>(src), lds, rows,
                  weights, (int)topk, tokens, chunks, static_cast<T*>(out), ldo);
}

template <typename T>
gemm_status_t gather(const void* src, int64_t lds, const int32_t* rows, const float* weights,
                     int64_t tokens, int64_t topk, int64_t hidden, void* out, int64_t ldo,
                     gemm_stream_t stream) {
    return (wide(hidden, {src, out}, {lds, ldo}) ? gather_v<T, 8> : gather_v<T, 1>)(
        src, lds, rows, weights, tokens, topk, hidden, out, ldo, stream);
}

template <typename T, int V>
gemm_status_t combine_grad_v(const void* dy, int64_t lddy, const void* ys, int64_t ldys, const int32_t* rows,
                             const int32_t* slots, const float* weights, int64_t tokens, int64_t topk,
                             int64_t hidden, void* dys, int64_t lddys, float* dweights, gemm_stream_t stream) {
    const int chunks = (int)(hidden / V);
    const int threads = (int)std::min<int64_t>(256, std::max<int64_t>(32, (chunks + 31) / 32 * 32));
    auto* fn = topk <= 2 ? combine_grad_kernel<T, V, 2> : combine_grad_kernel<T, V, 4>;
    return launch(fn, tokens, threads, 0, stream, static_cast<const T*>(dy), lddy, static_cast<const T*>(ys),
                  ldys, rows, slots, weights, (int)topk, tokens, chunks, static_cast<T*>(dys), lddys, dweights);
}

template <typename T>
gemm_status_t combine_grad(const void* dy, int64_t lddy, const void* ys, int64_t ldys, const int32_t* rows,
                           const int32_t* slots, const float* weights, int64_t tokens, int64_t topk,
                           int64_t hidden, void* dys, int64_t lddys, float* dweights, gemm_stream_t stream) {
    return (wide(hidden, {dy, ys, dys}, {lddy, ldys, lddys}) ? combine_grad_v<T, 8> : combine_grad_v<T, 1>)(
        dy, lddy, ys, ldys, rows, slots, weights, tokens, topk, hidden, dys, lddys, dweights, stream);
}

template <typename I>
gemm_status_t sort(const void* ids, int64_t ld, const SortArgs& shape, int32_t* offsets, int32_t* rows,
                   int32_t* slots, void* workspace, gemm_stream_t stream) {
    SortArgs a = shape;
    a.ld = ld;
    uint32_t* table = static_cast<uint32_t*>(workspace);
    if (a.blocks > 1) {
        const gemm_status_t st = launch(count_kernel<I>, a.blocks, 1024, 0, stream, static_cast<const I*>(ids), a, table);
        if (st != GEMM_OK) return st;
    }
    // a warp handles 128 slots of a full chunk; a short one takes fewer warps
    const int threads = a.total > 1024 ? 1024 : 256;
    if (threads == 256) a.chunk = 1024;
    const size_t smem = (size_t)threads / 32 * a.experts * sizeof(uint32_t);
    if (smem > 32 * 1024 && cudaFuncSetAttribute((const void*)place_kernel<I>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)smem) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    return launch(place_kernel<I>, a.blocks, threads, smem, stream, static_cast<const I*>(ids), a, table,
                  offsets, rows, slots);
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
    if (st != GEMM_OK) return st;
    const SortArgs a = sort_shape(tokens, topk, experts);
    *bytes = a.blocks > 1 ? (size_t)a.blocks * a.experts * sizeof(uint32_t) : 0;
    return GEMM_OK;
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
    const SortArgs a = sort_shape(tokens, topk, experts);
    if (a.blocks > 1 && (!workspace || misaligned(workspace, 16))) return GEMM_ERR_WORKSPACE;
    return (id_type == GEMM_INDEX_I64 ? sort<int64_t> : sort<int32_t>)(ids, ld_ids, a, offsets, rows, slots,
                                                                       workspace, stream);
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
    // a copy: the type does not matter
    const bool w = wide(hidden, {x, xs}, {ldx, ldxs});
    const int chunks = (int)(w ? hidden / 8 : hidden);
    return launch(w ? dispatch_kernel<__half, 8> : dispatch_kernel<__half, 1>, blocks_for(tokens * chunks), 256, 0,
                  stream, static_cast<const __half*>(x), ldx, rows, slots, (int)topk, tokens, chunks,
                  static_cast<__half*>(xs), ldxs);
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
    return (dtype == GEMM_BF16 ? combine_grad<__nv_bfloat16> : combine_grad<__half>)(
        dy, lddy, ys, ldys, rows, slots, weights, tokens, topk, hidden, dys, lddys, dweights, stream);
}

}  // extern "C"
