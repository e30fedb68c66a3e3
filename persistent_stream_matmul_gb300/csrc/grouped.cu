// Grouped products of include/gemm_moe.h: plans, tensor maps, launches and the
// C entry points.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <chrono>
#include <mutex>
#include <new>

#include "gemm_moe.h"
#include "grouped_kernel.cuh"

using namespace psm;

static_assert(G_MAX_GROUPS == GEMM_MOE_MAX_EXPERTS, "the kernel's tables hold every group");

struct gemm_grouped_plan {
    int64_t groups, rows, N, K;
    int kind, dtype, layout_b, device, num_sms;
    bool offline;
    int opt_ctas;
    // derived
    int ctas;             // CTAs of a scheduling unit
    int64_t m_total;      // C's contiguous extent (the lanes side)
    GroupedShape shape;
    size_t counter_bytes, ws_bytes;
    int* d_status;        // G_WORDS words
    int timeouts;         // G_WORD_TIMEOUTS
};

namespace {

constexpr int64_t MAX_INDEX = (1ll << 31) - 1024;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// Run numbers tagged into the split tiles' counters, 48 bits, unique in the
// process and started from the clock, so that what another run or program left
// in a workspace is not taken for this run's.
uint64_t next_epoch() {
    static std::atomic<uint64_t> epoch{
        (uint64_t)std::chrono::steady_clock::now().time_since_epoch().count() << 8};
    uint64_t e;
    do e = ++epoch & 0xffffffffffffull;
    while (e == 0);
    return e;
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

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Kernels, by [pair][ROWS K-major, ROWS MN-major, INNER][bf16].
template <bool PAIR>
void* kernel_of(int form, bool bf16) {
    switch (form) {
        case 0: return bf16 ? (void*)&grouped_kernel<PAIR, false, false, true> : (void*)&grouped_kernel<PAIR, false, false, false>;
        case 1: return bf16 ? (void*)&grouped_kernel<PAIR, false, true, true> : (void*)&grouped_kernel<PAIR, false, true, false>;
        default: return bf16 ? (void*)&grouped_kernel<PAIR, true, true, true> : (void*)&grouped_kernel<PAIR, true, true, false>;
    }
}

int smem_of(int ctas) { return ctas == 2 ? GroupedCfg<true>::SMEM_BYTES : GroupedCfg<false>::SMEM_BYTES; }

// The kernel of a plan with its shared memory allowed on the current device;
// null when that fails.
void* prepared_kernel(int ctas, int form, bool bf16, int dev) {
    static std::mutex mu;
    static bool ready[64][2][3][2];
    void* fn = ctas == 2 ? kernel_of<true>(form, bf16) : kernel_of<false>(form, bf16);
    if (dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    bool& r = ready[dev][ctas - 1][form][bf16];
    if (!r) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(ctas)) != cudaSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        r = true;
    }
    return fn;
}

// Pairs of CTAs that can be resident at once: a cluster lives inside one GPC,
// so this can be below #SMs / 2.  0 when unknown.
int resident_pairs(int dev) {
    static std::mutex mu;
    static int cache[64];
    void* fn = prepared_kernel(2, 0, true, dev);
    if (!fn) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev]) return cache[dev];
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(G_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem_of(2);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return cache[dev] = n;
}

gemm_status_t derive(gemm_grouped_plan* p) {
    const bool inner = p->kind == GEMM_GROUPED_INNER;
    const bool col = p->layout_b == GEMM_COL_MAJOR;
    // the lanes side is C's contiguous dimension
    p->m_total = inner && col ? p->K : p->N;
    const int64_t n_total = inner ? (col ? p->N : p->K) : 0;
    int ctas = p->opt_ctas;
    if (ctas == 0) {
        // Pairs halve the reads of Q and P a multiplication and store longer runs:
        // they win when there are rows enough for the tensor cores (INNER: always)
        // and tiles for all pairs.  us, one CTA against a pair: ROWS 64 groups of
        // 2048 x 1536, 128 rows each 79.4 / 78.6, 512 rows 178 / 138; one group of
        // 4096 x 4096, 256 rows (16 pair tiles) 16.4 / 21.2, 1024 rows (64) 32.2 /
        // 24.6; 16 groups of 512 x 512, 512 rows (64 tiles of 8 k-blocks) 9.0 / 9.5.
        // INNER 64 groups of 2048 x 1536, 32 rows 103 / 83, 512 rows 210 / 141; 16
        // groups of 512 x 512 (64 pair tiles), 32 rows 6.6 / 7.4.
        const bool wide = p->m_total > 128 && (!inner || n_total > 128);
        const int64_t pair_tiles = cdiv(p->m_total, 256) * (inner ? p->groups * cdiv(n_total, 256) : cdiv(p->rows, 256));
        const bool enough = inner ? 2 * pair_tiles > p->num_sms : p->rows > 128 * p->groups && pair_tiles >= 64;
        ctas = wide && enough ? 2 : 1;
    }
    const int tile = 128 * ctas;
    GroupedShape s{};
    s.groups = (int32_t)p->groups;
    s.rows = (int32_t)p->rows;
    s.inner = inner;
    s.tiles_m = (int32_t)cdiv(p->m_total, tile);
    s.tiles_n = (int32_t)cdiv(n_total, tile);
    s.n_total = (int32_t)n_total;
    s.kb = inner ? 0 : (int32_t)cdiv(p->K, G_BK);
    s.tile_n = tile;
    s.tile_shift = ctas == 2 ? 8 : 7;
    s.step = 16 * ctas;
    // a round of 76 pairs in a band of b tiles reads b + 76 / b operand tiles,
    // least near 9 (with 4, 16384 rows of 14336 x 4096 took 1252 us against 1214)
    s.band = 8;
    s.least_share = ctas == 2 ? 24 : 20;
    s.units = p->num_sms / ctas;
    if (ctas == 2 && !p->offline) {
        const int n = resident_pairs(p->device);
        if (n > 0) s.units = std::min(s.units, n);
    }
    const int64_t tiles_n = inner ? p->groups * s.tiles_n : p->rows / tile + std::min(p->groups, p->rows);
    if (s.tiles_m > 0 && tiles_n > MAX_INDEX / s.tiles_m) return GEMM_ERR_UNSUPPORTED;
    const int64_t k_blocks = inner ? s.tiles_m * s.tiles_n * (p->rows / G_BK + p->groups) : (int64_t)s.units * s.kb;
    s.may_split = k_blocks < MAX_INDEX && (!inner || tiles_n * s.tiles_m < s.units);
    p->ctas = ctas;
    p->shape = s;
    p->counter_bytes = p->ws_bytes = 0;
    if (s.may_split && p->rows > 0 && p->K > 0 && p->N > 0) {
        // fewer tiles than units are split: a counter a tile and CTA, a partial slot a CTA
        const size_t slot = 128 * (size_t)tile * sizeof(float), grid = (size_t)s.units * ctas;
        p->counter_bytes = (grid * 8 + 255) / 256 * 256;
        p->ws_bytes = p->counter_bytes + grid * slot;
    }
    return GEMM_OK;
}

gemm_status_t make_plan(gemm_grouped_plan_t* out, int kind, int64_t groups, int64_t rows, int64_t N,
                        int64_t K, int dtype, int layout_b, bool offline, int num_sms) {
    if (!out || groups < 1 || rows < 0 || N < 0 || K < 0 ||
        (kind != GEMM_GROUPED_ROWS && kind != GEMM_GROUPED_INNER) ||
        (dtype != GEMM_F16 && dtype != GEMM_BF16) ||
        (layout_b != GEMM_ROW_MAJOR && layout_b != GEMM_COL_MAJOR) || (offline && num_sms < 2))
        return GEMM_ERR_INVALID_ARG;
    if (groups > GEMM_MOE_MAX_EXPERTS || rows > MAX_INDEX || N > MAX_INDEX || K > MAX_INDEX || N % 8 || K % 8)
        return GEMM_ERR_UNSUPPORTED;
    int dev = -1;
    if (!offline) {
        int count = 0, major = 0, minor = 0;
        if (cudaGetDeviceCount(&count) != cudaSuccess || count == 0) {
            cudaGetLastError();
            return GEMM_ERR_NO_DEVICE;
        }
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return GEMM_ERR_CUDA;
        if (major != 10 || minor != 3) return GEMM_ERR_NO_DEVICE;
    }
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
    p->num_sms = num_sms;
    p->offline = offline;
    const gemm_status_t st = derive(p);
    if (st != GEMM_OK) {
        delete p;
        return st;
    }
    if (!offline && (cudaMalloc(&p->d_status, G_WORDS * sizeof(int)) != cudaSuccess ||
                     cudaMemset(p->d_status, 0, G_WORDS * sizeof(int)) != cudaSuccess)) {
        cudaGetLastError();
        if (p->d_status) cudaFree(p->d_status);
        delete p;
        return GEMM_ERR_CUDA;
    }
    *out = p;
    return GEMM_OK;
}

// 128-byte-swizzled map of a matrix stack: dims {x, y, z}, rows of ld elements.
bool encode(CUtensorMap* m, int dtype, const void* base, int rank, int64_t x, int64_t y, int64_t z,
            uint32_t box_x, uint32_t box_y) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)x, (cuuint64_t)y, (cuuint64_t)z};
    const cuuint64_t strides[2] = {(cuuint64_t)x * 2, (cuuint64_t)x * (cuuint64_t)y * 2};
    const cuuint32_t box[3] = {box_x, box_y, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, dtype == GEMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
               (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

gemm_status_t gemm_grouped_plan_create(gemm_grouped_plan_t* out, gemm_grouped_kind_t kind,
                                       int64_t groups, int64_t rows, int64_t N, int64_t K,
                                       gemm_dtype_t dtype, gemm_layout_t layout_b) {
    return make_plan(out, kind, groups, rows, N, K, dtype, layout_b, false, 0);
}

gemm_status_t gemm_grouped_plan_create_offline(gemm_grouped_plan_t* out, gemm_grouped_kind_t kind,
                                               int64_t groups, int64_t rows, int64_t N, int64_t K,
                                               gemm_dtype_t dtype, gemm_layout_t layout_b,
                                               int num_sms) {
    return make_plan(out, kind, groups, rows, N, K, dtype, layout_b, true, num_sms);
}

gemm_status_t gemm_grouped_plan_set_option(gemm_grouped_plan_t p, int key, int64_t value) {
    if (!p || (key != GEMM_GROUPED_OPT_CTAS && key != GEMM_GROUPED_OPT_INJECT_GIVE_UP)) return GEMM_ERR_INVALID_ARG;
    if (key == GEMM_GROUPED_OPT_INJECT_GIVE_UP) {
        if (value < -1 || value >= p->shape.units) return GEMM_ERR_UNSUPPORTED;
        if (p->offline) return GEMM_ERR_NO_DEVICE;
        DeviceGuard guard(p->device);
        const int word = (int)value + 1;
        return guard.ok && cudaMemcpy(p->d_status + G_WORD_GIVE_UP, &word, sizeof(int), cudaMemcpyHostToDevice) == cudaSuccess
                   ? GEMM_OK
                   : GEMM_ERR_CUDA;
    }
    if (value < 0 || value > 2) return GEMM_ERR_UNSUPPORTED;
    const int saved = p->opt_ctas;
    p->opt_ctas = (int)value;
    const gemm_status_t st = derive(p);
    if (st != GEMM_OK) {
        p->opt_ctas = saved;
        derive(p);
    }
    return st;
}

gemm_status_t gemm_grouped_plan_get_info(gemm_grouped_plan_t p, int key, int64_t* value) {
    if (!p || !value) return GEMM_ERR_INVALID_ARG;
    switch (key) {
        case GEMM_GROUPED_INFO_CTAS: *value = p->ctas; break;
        case GEMM_GROUPED_INFO_UNITS: *value = p->shape.units; break;
        case GEMM_GROUPED_INFO_TILE_M: *value = 128 * p->ctas; break;
        case GEMM_GROUPED_INFO_TILE_N: *value = p->shape.tile_n; break;
        case GEMM_GROUPED_INFO_STAGES: *value = GroupedCfg<true>::STAGES; break;
        case GEMM_GROUPED_INFO_SMEM_BYTES: *value = smem_of(p->ctas); break;
        case GEMM_GROUPED_INFO_GROUPS: *value = p->groups; break;
        default: return GEMM_ERR_INVALID_ARG;
    }
    return GEMM_OK;
}

gemm_status_t gemm_grouped_plan_units(gemm_grouped_plan_t p, const int32_t* offsets, int64_t unit,
                                      int32_t* units, int64_t max_units, int64_t* n_units) {
    if (!p || !offsets || !n_units || unit < 0 || unit >= p->shape.units || max_units < 0 ||
        (max_units > 0 && !units))
        return GEMM_ERR_INVALID_ARG;
    const GroupedShape& s = p->shape;
    int32_t first[G_MAX_GROUPS + 1];
    if (offsets[0] < 0 || offsets[s.groups] > s.rows) return GEMM_ERR_INVALID_ARG;
    for (int g = 0; g < s.groups; ++g)
        if (offsets[g + 1] < offsets[g]) return GEMM_ERR_INVALID_ARG;
    int32_t blocks = 0;
    auto fill = [&](int32_t most) {
        first[0] = 0;
        for (int g = 0; g < s.groups; ++g) {
            const int32_t n = offsets[g + 1] - offsets[g], kb = grouped_k_blocks(s, n);
            if (most == 0 && s.may_split) blocks += s.inner ? grouped_tiles(s, n) * kb : 0;
            first[g + 1] = first[g] + grouped_tiles(s, n) * grouped_shares(kb, most);
        }
    };
    fill(0);
    const GroupedSplit split = grouped_split(s, first[s.groups], blocks);
    if (s.inner && split.most > 0) fill(split.most);
    const GroupedTables tab{offsets, first};
    GroupedWork w;
    int64_t n = 0;
    for (; grouped_work(s, tab, split, (int32_t)unit, (int32_t)n, first[s.groups], w); ++n) {
        if (n >= max_units) continue;
        const int32_t v[9] = {w.shares > 1 ? -1 - w.item : w.item, w.group, w.tm, w.n0, w.valid, w.width, w.k0, w.k1, w.kb};
        std::copy(v, v + 9, units + 9 * n);
    }
    *n_units = n;
    return GEMM_OK;
}

gemm_status_t gemm_grouped_workspace_size(gemm_grouped_plan_t p, size_t* bytes) {
    if (!p || !bytes) return GEMM_ERR_INVALID_ARG;
    *bytes = p->ws_bytes;
    return GEMM_OK;
}

gemm_status_t gemm_grouped_run(gemm_grouped_plan_t p, const void* A, const void* B, void* C,
                               const int32_t* offsets, void* workspace, gemm_stream_t stream) {
    if (!p) return GEMM_ERR_INVALID_ARG;
    if (p->offline) return GEMM_ERR_NO_DEVICE;
    const bool inner = p->kind == GEMM_GROUPED_INNER;
    if (p->N == 0 || (inner ? p->K : p->rows) == 0) return GEMM_OK;  // C is empty
    const bool sums = inner ? p->rows > 0 : p->K > 0;                // something to sum
    if (!C || !offsets || (sums && (!A || !B))) return GEMM_ERR_INVALID_ARG;
    if (((uintptr_t)A & 15u) || ((uintptr_t)B & 15u) || ((uintptr_t)C & 15u) || ((uintptr_t)offsets & 3u))
        return GEMM_ERR_UNSUPPORTED;
    if (p->ws_bytes > 0 && (!workspace || ((uintptr_t)workspace & 15u))) return GEMM_ERR_WORKSPACE;
    DeviceGuard guard(p->device);
    if (!guard.ok) return GEMM_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!sums) {  // empty sums: +0
        const size_t bytes = 2 * (size_t)p->N * (size_t)(inner ? p->groups * p->K : p->rows);
        return cudaMemsetAsync(C, 0, bytes, st) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
    }
    const bool bf16 = p->dtype == GEMM_BF16, col = p->layout_b == GEMM_COL_MAJOR;
    const int form = inner ? 2 : (col ? 0 : 1);
    void* fn = prepared_kernel(p->ctas, form, bf16, p->device);
    if (!fn) return GEMM_ERR_CUDA;

    // The maps are encoded for every run: they cost well under a microsecond
    // of host time, and nothing is kept by an operand's address.
    GroupedMaps<false> tm_rows;
    GroupedMaps<true> tm_inner;
    bool ok = true;
    if (inner) {
        const void* P = col ? A : B;  // C's contiguous dimension
        const void* Q = col ? B : A;
        for (int i = 0; i < 7; ++i)
            ok = ok && encode(&tm_inner.p[i], p->dtype, P, 2, p->m_total, p->rows, 1, 64, 1u << i) &&
                 encode(&tm_inner.q[i], p->dtype, Q, 2, p->shape.n_total, p->rows, 1, 64, 1u << i);
        ok = ok && encode(&tm_inner.c, p->dtype, C, 3, p->m_total, p->shape.n_total, p->groups, 64, 32);
    } else {
        ok = col ? encode(&tm_rows.p[0], p->dtype, B, 3, p->K, p->N, p->groups, G_BK, 128)
                 : encode(&tm_rows.p[0], p->dtype, B, 3, p->N, p->K, p->groups, 64, G_BK);
        for (int i = 0; i < 4; ++i)
            ok = ok && encode(&tm_rows.q[i], p->dtype, A, 2, p->K, p->rows, 1, G_BK, 16u << i);
        ok = ok && encode(&tm_rows.c, p->dtype, C, 3, p->m_total, p->rows, 1, 64, 32);
    }
    if (!ok) return GEMM_ERR_UNSUPPORTED;

    GroupedParams kp{};
    kp.s = p->shape;
    kp.m_total = (int32_t)p->m_total;
    kp.out_group = p->N * p->K;
    kp.out = C;
    kp.offsets = offsets;
    if (p->ws_bytes > 0) {
        kp.counters = reinterpret_cast<unsigned long long*>(workspace);
        kp.partials = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + p->counter_bytes);
    }
    kp.epoch = next_epoch();
    kp.status = p->d_status;
    kp.idesc = idesc_f16(bf16, inner || !col, inner, 128 * p->ctas, 0);
    // a wait may last as long as the longest tile's k-loop
    kp.pipe_limit_ns = 4000000000ull + 2000ull * (uint64_t)cdiv(inner ? p->rows : p->K, G_BK);

    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p->shape.units * p->ctas), 1, 1);
    cfg.blockDim = dim3(G_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem_of(p->ctas);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    unsigned na = 0;
    if (p->ctas == 2) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = 2;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
    cfg.attrs = attr;
    cfg.numAttrs = na;
    void* args[2] = {inner ? (void*)&tm_inner : (void*)&tm_rows, &kp};
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

gemm_status_t gemm_grouped_last_status(gemm_grouped_plan_t p, gemm_stream_t stream) {
    if (!p) return GEMM_ERR_INVALID_ARG;
    if (p->offline) return GEMM_ERR_NO_DEVICE;
    DeviceGuard guard(p->device);
    if (!guard.ok) return GEMM_ERR_CUDA;
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return GEMM_ERR_CUDA;
    int h = 0;
    if (cudaMemcpy(&h, p->d_status + G_WORD_STATUS, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return GEMM_ERR_CUDA;
    if (h == 0) return GEMM_OK;
    // another tag from here on (grouped_tag), which no run on another stream may
    // see changing under way
    static_assert(G_WORD_STATUS == 0 && G_WORD_TIMEOUTS == 1, "both words are written at once");
    const int words[2] = {0, p->timeouts + 1};
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(p->d_status, words, sizeof(words), cudaMemcpyHostToDevice) != cudaSuccess)
        return GEMM_ERR_CUDA;
    ++p->timeouts;
    return GEMM_ERR_TIMEOUT;
}

gemm_status_t gemm_grouped_plan_destroy(gemm_grouped_plan_t p) {
    if (!p) return GEMM_OK;
    if (p->d_status) cudaFree(p->d_status);
    delete p;
    return GEMM_OK;
}

}  // extern "C"
