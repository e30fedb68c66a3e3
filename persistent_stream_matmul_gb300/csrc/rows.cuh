// What the row operators share: chunks of eight 16-bit elements of rows of any
// alignment, and their launches.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <initializer_list>

#include "gemm.h"
#include "host.cuh"

namespace psm {

__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

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

template <typename... P, typename... A>
inline gemm_status_t launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, gemm_stream_t stream,
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

inline bool misaligned(const void* p, size_t size) { return ((uintptr_t)p & (size - 1)) != 0; }

// Whether every row starts at a 16-byte boundary and holds whole chunks.  Rows
// without elements do, wherever they are: the aligned kernels then touch no
// row, while the others cut a first chunk at the written row's boundary.
inline bool aligned_rows(int64_t hidden, std::initializer_list<const void*> bases, std::initializer_list<int64_t> lds) {
    if (hidden == 0) return true;
    int64_t bits = hidden * 2;
    for (const void* b : bases) bits |= (int64_t)(uintptr_t)b;
    for (int64_t ld : lds) bits |= ld * 2;
    return (bits & 15) == 0;
}

}  // namespace psm
