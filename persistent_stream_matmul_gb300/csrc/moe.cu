// Mixture-of-experts row operators of include/gemm_moe.h: the stable sort of
// the slots by expert, and the row movements with their gradients.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>
#include <mutex>

#include "gemm_moe.h"
#include "ptx.cuh"

using namespace psm;

namespace {

constexpr int64_t MAX_INDEX = (1ll << 31) - 1024;
constexpr int64_t MAX_TOPK = 65535;
constexpr int64_t MAX_HIDDEN = 1ll << 30;

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
// Up to this many slots one block does it all: us against two launches, 1024
// slots of 64 experts 3.6 / 4.6, 4096 of 256 8.0 / 7.8 (and the second launch's
// cost on the host), 8192 of 64 11.2 / 7.6.
constexpr int SORT_SINGLE = 4096;
// Else slots a block: 2048 while there are at most 64 blocks, then 4096 until
// there are SORT_BLOCKS, then an even part.  Every block reads all blocks'
// counts: 32768 slots of 64 experts take 7.9 us with 2048 and 9.7 with 4096,
// 262144 of 256 experts 12.0 and 11.4.
constexpr int SORT_CHUNK = 2048;
constexpr int SORT_BLOCKS = 128;
constexpr int SORT_BATCH = 8;      // slots a lane in flight

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
    for (int64_t b = s0 + threadIdx.x; b < s1; b += 4 * blockDim.x) {
        int e[4];  // four loads in flight
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = b + i * blockDim.x < s1 ? key_of(ids, a, b + i * blockDim.x) : a.experts;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e[i] < a.experts) atomicAdd(&hist[e[i]], 1u);
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
    // This block's counts by warp, SORT_BATCH slots a lane loaded ahead.  A slot's
    // place among its warp's slots of the same expert is the count so far and
    // the equal keys in lower lanes.  The lanes with an equal key come from one
    // ballot a key bit; __match_any_sync took about three times as long.
    int bits = 1;
    while ((1 << bits) <= E) ++bits;
    int key[SORT_BATCH];
    uint32_t place[SORT_BATCH];
    auto count_batch = [&](int64_t b) {
#pragma unroll
        for (int i = 0; i < SORT_BATCH; ++i) {
            const int64_t s = b + i * 32 + lane;
            key[i] = s < w1 ? key_of(ids, a, s) : E;
        }
#pragma unroll
        for (int i = 0; i < SORT_BATCH; ++i) {
            if (b + i * 32 >= w1) break;
            unsigned same = 0xffffffffu;
            for (int bit = 0; bit < bits; ++bit) {
                const unsigned ones = __ballot_sync(0xffffffffu, (key[i] >> bit) & 1);
                same &= (key[i] >> bit) & 1 ? ones : ~ones;
            }
            const uint32_t at = key[i] < E ? own[key[i]] : 0;
            place[i] = at + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (key[i] < E && lane == __ffs(same) - 1) own[key[i]] = at + __popc(same);
            __syncwarp();
        }
    };
    for (int64_t b = w0; b < w1; b += 32 * SORT_BATCH) count_batch(b);
    // all blocks' counts, and those of the blocks before this one
    if (a.blocks > 1) {
        const int parts = max(1, (int)blockDim.x / E);
        for (int i = threadIdx.x; i < parts * E; i += blockDim.x) {
            const int e = i % E;
            uint32_t sum = 0, prior = 0;
#pragma unroll 8
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
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            uint32_t sum = 0;
#pragma unroll 8
            for (int w = 0; w < warps; ++w) sum += mine[w * E + e];
            all[e] = sum;
        }
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
            for (int w = 0; w < warps; w += 8) {  // warps is a multiple of 8
                uint32_t n[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) n[i] = mine[(w + i) * E + e];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    mine[(w + i) * E + e] = at;
                    at += n[i];
                }
            }
            if (blockIdx.x == 0) offsets[e] = (int32_t)first;
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = (int32_t)carry;
    // place: own[e] now holds the warp's first row of expert e
    const bool one_batch = w1 - w0 <= 32 * SORT_BATCH;  // its keys and places are still here
    for (int64_t b = w0; b < w1; b += 32 * SORT_BATCH) {
        if (!one_batch) count_batch(b);  // advances own, so that places are rows
#pragma unroll
        for (int i = 0; i < SORT_BATCH; ++i) {
            const int64_t s = b + i * 32 + lane;
            if (key[i] < E) {
                const uint32_t r = one_batch ? own[key[i]] + place[i] : place[i];
                rows[s] = (int32_t)r;
                slots[r] = (int32_t)s;
            } else if (s < w1) {
                rows[s] = -1;
            }
        }
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
    if (a.total <= SORT_SINGLE) a.chunk = std::max<int64_t>(1024, (a.total + 1023) / 1024 * 1024);
    else if (a.total <= 64 * SORT_CHUNK) a.chunk = SORT_CHUNK;
    else a.chunk = std::max<int64_t>(2 * SORT_CHUNK, (even + 1023) / 1024 * 1024);
    a.blocks = (int)((a.total + a.chunk - 1) / a.chunk);
    if (a.blocks < 1) a.blocks = 1;
    return a;
}

// ---------------------------------------------------------------- row movements
// Bound by memory: every row is read or written once, 16 bytes a thread and
// access.  A group of whole warps takes a row (blockDim = width x rows a
// block), each thread C chunks of eight elements of it, strided by `width`,
// and U rows at a time, B blocks of 256 an SM.  What counts is the bytes in
// flight an SM, so U and C are weighed against the registers that B allows:
// the sum of 2 choices of 16384 tokens of 4096 takes 68 us with U, C, B = 2, 1, 4
// (5.9 TB/s), 71 with 2, 2, 4, 84 with 4, 1, 4 and 115 with 2, 2, 6, whose
// registers spill in the loop (before the streaming stores below, with which the
// first takes 63).
//
// ALIGNED: every row starts at a 16-byte boundary and its length is a multiple
// of 8.  Otherwise the chunks are cut at the 16-byte boundaries of the row
// that is written, so its inner chunks are stored whole, and a chunk of
// another row is put together from the two aligned 16-byte words that hold it
// (words without an element of the row are not read).
struct alignas(16) Chunk {
    uint32_t w[4];
};

// STREAM: read once; else the neighbouring thread's chunk shares the word.
// (Plain loads, not the read-only path: the grid may have started before the
// kernel that wrote the rows ended.)
template <bool STREAM>
__device__ __forceinline__ Chunk load_word(const void* p) {
    const uint4* q = static_cast<const uint4*>(p);
    const uint4 x = STREAM ? __ldcs(q) : *q;
    return Chunk{{x.x, x.y, x.z, x.w}};
}

// Elements h .. h + 7 of a row of n; those outside [0, n) are unspecified.
template <bool ALIGNED>
__device__ __forceinline__ Chunk load_chunk(const uint16_t* row, int h, int n) {
    if constexpr (ALIGNED) return load_word<true>(row + h);
    const uintptr_t at = reinterpret_cast<uintptr_t>(row) + 2 * (int64_t)h;
    const int s = (int)(at >> 1) & 7;  // elements of the first word before the chunk
    const char* word = reinterpret_cast<const char*>(at - 2 * s);
    uint32_t w[8] = {};
    if (h + 8 - s > 0 && h < n) {
        const Chunk a = load_word<false>(word);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = a.w[i];
    }
    if (s > 0 && h + 8 > 0 && h + 8 - s < n) {
        const Chunk b = load_word<false>(word + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 + i] = b.w[i];
    }
    if (s & 1) {
#pragma unroll
        for (int i = 0; i < 7; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        w[7] >>= 16;
    }
    if (s & 2)
#pragma unroll
        for (int i = 0; i < 7; ++i) w[i] = w[i + 1];
    if (s & 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = w[i + 2];
    return Chunk{{w[0], w[1], w[2], w[3]}};
}

// Whole rows are written once and leave L2 first: 4 choices of 16384 tokens of
// 4096 108 -> 102 us, their gradient 191 -> 178.  Rows cut at other boundaries
// share their lines with their neighbours, which then wait in L2 (with the same
// hint, 18 -> 26 us for 16388 rows of 2047).
template <bool ALIGNED>
__device__ __forceinline__ void store_chunk(uint16_t* row, int h, int n, const Chunk& c) {
    if constexpr (ALIGNED) {
        __stcs(reinterpret_cast<uint4*>(row + h), make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]));
    } else if (h >= 0 && h + 8 <= n) {
        *reinterpret_cast<uint4*>(row + h) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (h + i >= 0 && h + i < n) row[h + i] = (uint16_t)(c.w[i / 2] >> (16 * (i & 1)));
    }
}

// Elements of the row at `row` before its first 16-byte boundary cut, 0 .. 7:
// chunk c of the row starts at element 8c - lead.
template <bool ALIGNED>
__device__ __forceinline__ int lead_of(const uint16_t* row) {
    return ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(row) >> 1) & 7;
}

template <typename T>
__device__ __forceinline__ void unpack(const Chunk& c, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w = c.w[i];
        const T* e = reinterpret_cast<const T*>(&w);
        x[2 * i] = to_f(e[0]);
        x[2 * i + 1] = to_f(e[1]);
    }
}

template <typename T>
__device__ __forceinline__ Chunk pack(const float (&x)[8]) {
    Chunk c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        T e[2] = {from_f<T>(x[2 * i]), from_f<T>(x[2 * i + 1])};
        c.w[i] = *reinterpret_cast<uint32_t*>(e);
    }
    return c;
}

// A row index out of range counts as dropped.
__device__ __forceinline__ int64_t row_at(const int32_t* rows, int64_t s, int64_t total) {
    const int64_t r = rows[s];
    return r >= 0 && r < total ? r : -1;
}

// out[rows[t, j]] = x[t], a token a thread group: x is read once (or, not
// aligned, once more from the cache for every choice, cut for its row).
template <bool ALIGNED, int C>
__global__ void __launch_bounds__(256)
    dispatch_kernel(const uint16_t* x, int64_t ldx, const int32_t* rows, const int32_t* slots, int topk,
                    int64_t tokens, int n, uint16_t* out, int64_t ldo) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, total = tokens * topk;
    if (t >= tokens) return;
    const uint16_t* src = x + t * ldx;
    const int width = blockDim.x, span = width * 8;
    for (int h0 = threadIdx.x * 8; h0 < n + (ALIGNED ? 0 : 7); h0 += span * C) {
        Chunk v[C];
        if constexpr (ALIGNED)
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (h0 + c * span < n) v[c] = load_chunk<true>(src, h0 + c * span, n);
        for (int j = 0; j < topk; ++j) {
            const int64_t s = t * topk + j, r = row_at(rows, s, total);
            if (r >= 0) {
                uint16_t* dst = out + r * ldo;
                const int lead = lead_of<ALIGNED>(dst);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int h = h0 + c * span - lead;
                    if constexpr (!ALIGNED)
                        if (h < n) v[c] = load_chunk<false>(src, h, n);
                }
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int h = h0 + c * span - lead;
                    if (h < n) store_chunk<ALIGNED>(dst, h, n, v[c]);
                }
            }
            if (slots[s] < 0) {  // row s is unused
                uint16_t* dst = out + s * ldo;
                const int lead = lead_of<ALIGNED>(dst);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int h = h0 + c * span - lead;
                    if (h < n) store_chunk<ALIGNED>(dst, h, n, Chunk{});
                }
            }
        }
    }
}

// out[t] = the sum over j of w[t, j] * src[rows[t, j]] (w NULL: 1), a token a
// thread group, in fp32 and ascending j.
template <typename T, bool ALIGNED, int U, int C, int B>
__global__ void __launch_bounds__(256, B)
    gather_kernel(const uint16_t* src, int64_t lds, const int32_t* rows, const float* weights, int topk,
                  int64_t tokens, int n, uint16_t* out, int64_t ldo) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, total = tokens * topk;
    if (t >= tokens) return;
    uint16_t* dst = out + t * ldo;
    const int lead = lead_of<ALIGNED>(dst);
    const int span = blockDim.x * 8;
    for (int h0 = threadIdx.x * 8 - lead; h0 < n; h0 += span * C) {
        float acc[C][8] = {};
        for (int j0 = 0; j0 < topk; j0 += U) {
            Chunk v[U][C];
            float w[U];
            bool use[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t s = t * topk + j0 + u;
                const int64_t r = j0 + u < topk ? row_at(rows, s, total) : -1;
                use[u] = r >= 0;
                if (use[u]) {
                    w[u] = weights ? weights[s] : 1.f;
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        if (h0 + c * span < n) v[u][c] = load_chunk<ALIGNED>(src + r * lds, h0 + c * span, n);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (use[u])
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        float x[8];
                        unpack<T>(v[u][c], x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[c][i] = fmaf(w[u], x[i], acc[c][i]);
                    }
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (h0 + c * span < n) store_chunk<ALIGNED>(dst, h0 + c * span, n, pack<T>(acc[c]));
    }
}

// dys[rows[t, j]] = w[t, j] * dy[t], and dweights[t, j] = dy[t] . ys[rows[t, j]],
// a token a thread group, U choices at a time (dy comes from the cache for the
// next U).  blockIdx.y takes every gridDim.y-th U.  A thread adds its chunks in
// ascending order, then the lanes and the warps are added in a fixed order.
template <typename T, bool ALIGNED, int U, int C, int B>
__global__ void __launch_bounds__(256, B)
    combine_grad_kernel(const uint16_t* dy, int64_t lddy, const uint16_t* ys, int64_t ldys, const int32_t* rows,
                        const int32_t* slots, const float* weights, int topk, int64_t tokens, int n,
                        uint16_t* dys, int64_t lddys, float* dweights) {
    __shared__ float part[U][8];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, total = tokens * topk;
    const bool in = t < tokens;
    const int span = blockDim.x * 8;
    const int warp = (threadIdx.y * blockDim.x + threadIdx.x) >> 5, warps = blockDim.x >> 5;
    const uint16_t* d = dy + t * lddy;
    for (int j0 = blockIdx.y * U; j0 < topk; j0 += gridDim.y * U) {
        float dot[U] = {};
        if (in) {
            int64_t r[U];
            float w[U];
            bool zero[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t s = t * topk + j0 + u;
                r[u] = j0 + u < topk ? row_at(rows, s, total) : -1;
                w[u] = r[u] >= 0 ? weights[s] : 0.f;
                zero[u] = j0 + u < topk && slots[s] < 0;
            }
            for (int h0 = threadIdx.x * 8; h0 < n + (ALIGNED ? 0 : 7); h0 += span * C) {
                constexpr int D = ALIGNED ? 1 : U;  // not aligned, dy is cut for each choice's row
                Chunk dv[D][C], yv[U][C];
                int lead[U];
#pragma unroll
                for (int u = 0; u < U; ++u) lead[u] = lead_of<ALIGNED>(dys + r[u] * lddys);
                if constexpr (ALIGNED)
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        if (h0 + c * span < n) dv[0][c] = load_chunk<true>(d, h0 + c * span, n);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (r[u] >= 0)
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            const int h = h0 + c * span - lead[u];
                            if (h < n) {
                                yv[u][c] = load_chunk<ALIGNED>(ys + r[u] * ldys, h, n);
                                if constexpr (!ALIGNED) dv[u][c] = load_chunk<false>(d, h, n);
                            }
                        }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const int h = h0 + c * span - lead[u];
                        if (r[u] >= 0 && h < n) {
                            float x[8], y[8], o[8];
                            unpack<T>(dv[ALIGNED ? 0 : u][c], x);
                            unpack<T>(yv[u][c], y);
                            if (!ALIGNED && (h < 0 || h + 8 > n))
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    if (h + i < 0 || h + i >= n) x[i] = y[i] = 0.f;  // not of the rows
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                o[i] = w[u] * x[i];
                                dot[u] = fmaf(x[i], y[i], dot[u]);
                            }
                            store_chunk<ALIGNED>(dys + r[u] * lddys, h, n, pack<T>(o));
                        }
                        if (zero[u]) {  // row t * topk + j is unused
                            uint16_t* dst = dys + (t * topk + j0 + u) * lddys;
                            const int z = h0 + c * span - lead_of<ALIGNED>(dst);
                            if (z < n) store_chunk<ALIGNED>(dst, z, n, Chunk{});
                        }
                    }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            for (int o = 16; o; o >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], o);
        if (warps > 1) {
            __syncthreads();  // the sums of the choices before have been read
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int u = 0; u < U; ++u) part[u][warp] = dot[u];
            __syncthreads();
        }
        if (in && threadIdx.x < U && j0 + (int)threadIdx.x < topk) {
            float sum = 0.f;
            if (warps > 1)
                for (int i = 0; i < warps; ++i) sum += part[threadIdx.x][threadIdx.y * warps + i];
            else
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if ((int)threadIdx.x == u) sum = dot[u];
            dweights[t * topk + j0 + threadIdx.x] = sum;
        }
    }
}

template <typename... P, typename... A>
gemm_status_t launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, gemm_stream_t stream,
                     A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.dynamicSmemBytes = smem;
    cfg.gridDim = grid;
    cfg.blockDim = block;
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
    if (topk > MAX_TOPK || tokens > MAX_INDEX / topk || hidden > MAX_HIDDEN) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// Whether every row starts at a 16-byte boundary and holds whole chunks.  Rows
// without elements do, wherever they are: the aligned kernels then touch no
// row, while the others cut a first chunk at the written row's boundary.
bool aligned_rows(int64_t hidden, std::initializer_list<const void*> bases, std::initializer_list<int64_t> lds) {
    if (hidden == 0) return true;
    int64_t bits = hidden * 2;
    for (const void* b : bases) bits |= (int64_t)(uintptr_t)b;
    for (int64_t ld : lds) bits |= ld * 2;
    return (bits & 15) == 0;
}

// Whole warps for a row, c chunks a thread, at most 256 threads (a longer row
// takes several even rounds), and as many rows a block as fit 256 threads.
dim3 row_block(int64_t hidden, int c) {
    const int64_t chunks = (hidden + 7) / 8;
    const int64_t rounds = std::max<int64_t>(1, (chunks + 256 * c - 1) / (256 * c));
    const int64_t threads = (chunks + rounds * c - 1) / (rounds * c);
    const unsigned width = (unsigned)std::max<int64_t>(32, (threads + 31) / 32 * 32);
    return dim3(width, width < 256 ? 256 / width : 1, 1);
}

dim3 row_grid(int64_t tokens, dim3 block, int64_t groups = 1) {
    return dim3((unsigned)((tokens + block.y - 1) / block.y), (unsigned)groups, 1);
}

template <typename T, bool ALIGNED, int U, int C, int B>
gemm_status_t gather_v(const void* src, int64_t lds, const int32_t* rows, const float* weights,
                       int64_t tokens, int64_t topk, int64_t hidden, void* out, int64_t ldo,
                       gemm_stream_t stream) {
    const dim3 block = row_block(hidden, C);
    return launch(gather_kernel<T, ALIGNED, U, C, B>, row_grid(tokens, block), block, 0, stream,
                  static_cast<const uint16_t*>(src), lds, rows, weights, (int)topk, tokens, (int)hidden,
                  static_cast<uint16_t*>(out), ldo);
}

template <typename T>
gemm_status_t gather(const void* src, int64_t lds, const int32_t* rows, const float* weights,
                     int64_t tokens, int64_t topk, int64_t hidden, void* out, int64_t ldo,
                     gemm_stream_t stream) {
    // us for rows of 4096 unless said.  1 choice: 44.5 with this, though 40 registers
    // spill 90 bytes a thread, 48.2 with B = 4 (6.9 and 6.7 for 4096 rows of 2048) and
    // 48.8 with the next.  4 choices: 102.4 with this, 103.2 with U, C = 4, 1 and 103.3
    // with 2, 1; rows of 1024 52.7, 56.0 and 55.2.  Not aligned, rows of 2047: 19.6,
    // with U = 2 20.6.
    auto* fn = !aligned_rows(hidden, {src, out}, {lds, ldo}) ? gather_v<T, false, 1, 1, 4>
               : topk == 1                                   ? gather_v<T, true, 1, 2, 6>
               : topk == 2                                   ? gather_v<T, true, 2, 1, 4>
                                                             : gather_v<T, true, 2, 2, 4>;
    return fn(src, lds, rows, weights, tokens, topk, hidden, out, ldo, stream);
}

template <typename T, bool ALIGNED, int U, int C, int B>
gemm_status_t combine_grad_v(const void* dy, int64_t lddy, const void* ys, int64_t ldys, const int32_t* rows,
                             const int32_t* slots, const float* weights, int64_t tokens, int64_t topk,
                             int64_t hidden, void* dys, int64_t lddys, float* dweights, gemm_stream_t stream) {
    const dim3 block = row_block(hidden, C);
    // U choices a thread group when the tokens alone would not fill the device
    // (us, one group after another against each its own block: 8 choices of 4096,
    // 16 tokens 5.6 / 3.5, 256 6.9 / 6.1, 1024 23.7 / 23.3)
    const int64_t groups = tokens <= 1024 ? (topk + U - 1) / U : 1;
    return launch(combine_grad_kernel<T, ALIGNED, U, C, B>, row_grid(tokens, block, groups), block, 0, stream,
                  static_cast<const uint16_t*>(dy), lddy, static_cast<const uint16_t*>(ys), ldys, rows, slots,
                  weights, (int)topk, tokens, (int)hidden, static_cast<uint16_t*>(dys), lddys, dweights);
}

template <typename T>
gemm_status_t combine_grad(const void* dy, int64_t lddy, const void* ys, int64_t ldys, const int32_t* rows,
                           const int32_t* slots, const float* weights, int64_t tokens, int64_t topk,
                           int64_t hidden, void* dys, int64_t lddys, float* dweights, gemm_stream_t stream) {
    // us with U, C, B = 4, 1, 4 (2, 1, 6 for 2 choices) against 2, 2, 4: 4 choices
    // of 4096 184 / 186 and 2 of them 98 / 107, but 6 of 4096 146 / 138, 8 of 2048
    // 96 / 92, 6 of 1080 76 / 70, 4 of 512 25.4 / 22.1, 2 of 1024 26.6 / 24.0
    auto* fn = !aligned_rows(hidden, {dy, ys, dys}, {lddy, ldys, lddys}) ? combine_grad_v<T, false, 1, 2, 4>
               : topk > 4 || hidden < 2048                               ? combine_grad_v<T, true, 2, 2, 4>
               : topk <= 2                                               ? combine_grad_v<T, true, 2, 1, 6>
                                                                         : combine_grad_v<T, true, 4, 1, 4>;
    return fn(dy, lddy, ys, ldys, rows, slots, weights, tokens, topk, hidden, dys, lddys, dweights, stream);
}

// Allows place_kernel all the shared memory that it may need on the current
// device, once: the limit is the function's, so a call that set its own size
// could lower it between another thread's setting and launch.
template <typename I>
bool place_memory_allowed() {
    static std::mutex mu;
    static bool ready[64];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return false;
    }
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
        constexpr int most = 32 * GEMM_MOE_MAX_EXPERTS * (int)sizeof(uint32_t);
        if (cudaFuncSetAttribute((const void*)place_kernel<I>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        ready[dev] = true;
    }
    return true;
}

template <typename I>
gemm_status_t sort(const void* ids, int64_t ld, const SortArgs& shape, int32_t* offsets, int32_t* rows,
                   int32_t* slots, void* workspace, gemm_stream_t stream) {
    SortArgs a = shape;
    a.ld = ld;
    uint32_t* table = static_cast<uint32_t*>(workspace);
    if (a.blocks > 1) {
        const gemm_status_t st = launch(count_kernel<I>, dim3(a.blocks), dim3(1024), 0, stream, static_cast<const I*>(ids), a, table);
        if (st != GEMM_OK) return st;
    }
    const int threads = a.total > 1024 ? 1024 : 256;
    const size_t smem = (size_t)threads / 32 * a.experts * sizeof(uint32_t);
    if (smem > 32 * 1024 && !place_memory_allowed<I>()) return GEMM_ERR_CUDA;
    return launch(place_kernel<I>, dim3(a.blocks), dim3(threads), smem, stream, static_cast<const I*>(ids), a, table,
                  offsets, rows, slots);
}

gemm_status_t check_sort(int64_t tokens, int64_t topk, int64_t experts) {
    if (tokens < 0 || topk < 1 || experts < 1) return GEMM_ERR_INVALID_ARG;
    if (experts > GEMM_MOE_MAX_EXPERTS || topk > MAX_TOPK || tokens > MAX_INDEX / topk)
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
    const bool al = aligned_rows(hidden, {x, xs}, {ldx, ldxs});
    const dim3 block = row_block(hidden, 4);
    return launch(al ? dispatch_kernel<true, 4> : dispatch_kernel<false, 4>, row_grid(tokens, block), block, 0, stream,
                  static_cast<const uint16_t*>(x), ldx, rows, slots, (int)topk, tokens, (int)hidden,
                  static_cast<uint16_t*>(xs), ldxs);
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
