// Scaled products of include/gemm_scaled.h: plans, tensor maps, launches and the
// C entry points.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>
#include <new>

#include "gemm_scaled.h"
#include "host.cuh"
#include "rows.cuh"
#include "scaled_few.cuh"

using namespace psm;

static_assert(S_BK == GEMM_SCALE_GROUP, "a k-block is a group");

struct gemm_scaled_plan {
    int64_t M, N, K;
    int type_a, type_b, out_dtype, layout_a, layout_b, scale_a, scale_b;
    int device, num_sms;
    bool offline;
    int opt_ctas, opt_form;
    // derived
    int form, ctas, turned, col_vector;
    ScaledShape shape;
    size_t counter_bytes, ws_bytes;
    int* d_status;           // G_WORDS words
    int timeouts;            // G_WORD_TIMEOUTS
};

namespace {

struct Kernel {
    void* fn;
    int smem, stages;
};

template <bool PAIR, bool TURNED, bool COL_VECTOR>
Kernel kernel_v() {
    using Cf = ScaledCfg<PAIR, TURNED, COL_VECTOR>;
    return {(void*)&scaled_kernel<PAIR, TURNED, COL_VECTOR>, Cf::SMEM_BYTES, Cf::STAGES};
}

Kernel kernel_of(int ctas, int turned, int col_vector) {
    if (turned) return kernel_v<false, true, true>();
    if (ctas == 2) return col_vector ? kernel_v<true, false, true>() : kernel_v<true, false, false>();
    return col_vector ? kernel_v<false, false, true>() : kernel_v<false, false, false>();
}

// Whether the kernel may use its shared memory on the current device.
bool prepared(int ctas, int turned, int col_vector, int dev) {
    static std::mutex mu;
    static bool ready[64][2][2][2];
    if (dev < 0 || dev >= 64) return false;
    const Kernel k = kernel_of(ctas, turned, col_vector);
    std::lock_guard<std::mutex> lock(mu);
    bool& r = ready[dev][ctas - 1][turned][col_vector];
    if (!r) {
        cudaFuncAttributes attr{};
        if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) != cudaSuccess ||
            cudaFuncGetAttributes(&attr, k.fn) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        // the epilogue of a pair waits for registers that the launch must have had
        if (ctas == 2 && attr.numRegs < S_REGS) return false;
        r = true;
    }
    return true;
}

// Pairs of CTAs that can be resident at once: a cluster lives inside one GPC,
// so this can be below #SMs / 2.  0: pairs cannot run.
int resident_pairs(int col_vector, int dev) {
    static std::mutex mu;
    static int cache[64][2];
    if (!prepared(2, 0, col_vector, dev)) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev][col_vector]) return cache[dev][col_vector];
    const Kernel k = kernel_of(2, 0, col_vector);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(S_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)k.smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k.fn, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return cache[dev][col_vector] = n;
}

gemm_status_t derive(gemm_scaled_plan* p) {
    const bool few = p->layout_a == GEMM_ROW_MAJOR && p->layout_b == GEMM_COL_MAJOR && cdiv(p->M, F_MOST_ROWS) <= 65535;
    // Without tensor memory: up to 16 rows always, more while the product is small. (us of 2, 8,
    // 12 and 16 rows, without against with: 14336 x 4096 14.2 / 15.7, 14.7 / 15.9, 17.8 / 16.0, 18.2 /
    // 15.9; 4096 x 14336 14.3 / 17.9, 14.4 / 18.0, 18.1 / 18.1, 18.3 / 18.2. So from 9 rows on it
    // loses up to 12 % on large matrices, and wins on smaller ones.) On tensor
    // memory it takes 5 us with few k-blocks and 8 to 12 with more, however small; without,
    // each 32 rows of A read B again and each 16 rows of B read those. us, without against
    // with: 24 x 1536 x 2048 3.6 / 9.3, 24 x 4096 x 4096 8.4 / 11.3, 32 x 4096 x 4096 10.5 /
    // 11.3, 64 x 2048 x 2048 6.0 / 8.5, 128 x 1024 x 1024 4.0 / 5.9, 128 x 256 x 8192 11.7 /
    // 12.4; but 256 x 1024 x 1024 6.9 / 6.0, 64 x 4096 x 512 5.7 / 4.9, 48 x 4096 x 2048 10.8 /
    // 9.1, 24 x 14336 x 4096 23.4 / 16.1.
    const double out = (double)p->M * (double)p->N, products = out * (double)p->K;
    const bool small = p->M <= 16 || (out <= 1.4e5 && products <= (p->M <= 32 ? 5.4e8 : 2.9e8));
    int form = p->opt_form, ctas = p->opt_ctas;
    // Turned, a tile's columns fit the rows of A, but each has a scale of its own to be
    // read and multiplied: us, turned against straight, 4096 x 14336 with 32 rows 18.6 /
    // 20.8, 4096 x 4096 with 17 rows 11.5 / 14.9, with 48 13.4 / 12.8, 14336 x 4096 with 64
    // 22.4 / 16.1.
    if (form < 0) form = ctas == 2 ? GEMM_SCALED_STRAIGHT : few && small ? GEMM_SCALED_FEW : p->M <= 32 ? GEMM_SCALED_TURNED : GEMM_SCALED_STRAIGHT;
    // Pairs read their operands half as often, single CTAs make four times the tiles: us,
    // single against pairs, 512 x 4096 x 4096 (32 pair tiles) 14.0 / 19.7, 256 x 14336 x
    // 4096 (56) 25.8 / 20.7, 1024 x 4096 x 4096 (64) 23.9 / 19.1. Where a round of the 76 pairs is
    // partly empty they are near: K of 1024, 1536, 4096 with 80 tiles 12.7 / 13.8, 16.7 / 17.2, 34.7 / 34.0,
    // with 112 12.9 / 14.1, 16.7 / 17.5, 36.0 / 35.5, with 144 15.9 / 15.0, 20.9 / 18.2, 46.1 / 35.0.
    if (ctas == 0) ctas = form == GEMM_SCALED_STRAIGHT && cdiv(p->M, 256) * cdiv(p->N, 256) >= 48 ? 2 : 1;
    if ((form != GEMM_SCALED_STRAIGHT && ctas == 2) || (form == GEMM_SCALED_FEW && !few)) return GEMM_ERR_UNSUPPORTED;
    const int turned = form != GEMM_SCALED_STRAIGHT, col_vector = turned || p->scale_b == GEMM_SCALE_VECTOR;
    const int pairs = ctas == 2 && !p->offline ? resident_pairs(col_vector, p->device) : 0;
    if (ctas == 2 && !p->offline && pairs == 0) {
        if (p->opt_ctas == 2) return GEMM_ERR_UNSUPPORTED;
        ctas = 1;
    }
    const int64_t lanes = turned ? p->N : p->M, cols = turned ? p->M : p->N;
    const int tile = 128 * ctas;
    ScaledShape s{};
    int64_t units = p->num_sms / ctas;
    if (pairs > 0) units = std::min<int64_t>(units, pairs);
    const int64_t tiles_l = cdiv(lanes, tile), side = cdiv(cols, tile), tiles = tiles_l * side, kb = cdiv(p->K, S_BK);
    if (tiles > MAX_INDEX) return GEMM_ERR_UNSUPPORTED;
    s.tiles = (int32_t)tiles;
    s.tiles_l = (int32_t)tiles_l;
    s.cols = (int32_t)cols;
    s.side = (int32_t)side;
    // straight tiles have one width, so that a half's columns share a block's scale
    const int64_t step = !turned ? tile : p->layout_a == GEMM_ROW_MAJOR ? 16 : 32;
    s.width = (int32_t)(cdiv(side == 0 ? 1 : cdiv(cols, side), step) * step);
    // even bands of about eight tiles along the columns side: a round of 76 pairs in a
    // band of b tiles reads b + 76 / b operand tiles, least near 9
    const int64_t bands = 2 * side > 24 ? (side + 3) / 8 : 1;
    s.band = (int32_t)cdiv(side, bands);
    s.kb = (int32_t)kb;
    s.units = (int32_t)units;
    // the tiles left over a whole round, in shares of `least` k-blocks at least: shorter
    // ones are not worth joining (us, single CTAs, with 12 and 16: 200 x 2048 x 2048 10.2 /
    // 8.4, 300 x 4096 x 2048 9.4 / 9.4; turned, 8 and 12: 24 x 4096 x 4096 11.5 / 11.6)
    const int64_t least = turned ? 8 : 16, rest = tiles < units ? tiles : tiles % units;
    s.shares = 1;
    if (rest > 0 && kb > least) {
        const int64_t most = std::max(cdiv(rest * kb, units - rest), least), shares = cdiv(kb, most);
        if (shares > 1) {
            s.split = (int32_t)rest;
            s.shares = (int32_t)shares;
        }
    }
    p->form = form;
    p->ctas = ctas;
    p->turned = turned;
    p->col_vector = col_vector;
    p->shape = s;
    p->counter_bytes = p->ws_bytes = 0;
    if (form != GEMM_SCALED_FEW && s.shares > 1) {
        const size_t slot = 128 * (size_t)tile * sizeof(float), grid = (size_t)s.units * ctas;
        p->counter_bytes = (grid * 8 + 255) / 256 * 256;
        p->ws_bytes = p->counter_bytes + grid * slot;
    }
    return GEMM_OK;
}

bool bad(int v) { return v != 0 && v != 1; }

gemm_status_t make_plan(gemm_scaled_plan_t* out, int64_t M, int64_t N, int64_t K, int type_a, int type_b, int out_dtype,
                        int layout_a, int layout_b, int scale_a, int scale_b, bool offline, int num_sms) {
    if (!out || M < 0 || N < 0 || K < 0 || bad(type_a) || bad(type_b) || bad(layout_a) || bad(layout_b) || bad(scale_a) ||
        bad(scale_b) || (out_dtype != GEMM_F16 && out_dtype != GEMM_BF16 && out_dtype != GEMM_F32) || (offline && num_sms < 2))
        return GEMM_ERR_INVALID_ARG;
    if (M > MAX_INDEX || N > MAX_INDEX || K > MAX_INDEX || (layout_a == GEMM_ROW_MAJOR ? K : M) % 16 ||
        (layout_b == GEMM_COL_MAJOR ? K : N) % 16)
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
    gemm_scaled_plan* p = new (std::nothrow) gemm_scaled_plan();
    if (!p) return GEMM_ERR_CUDA;
    p->M = M;
    p->N = N;
    p->K = K;
    p->type_a = type_a;
    p->type_b = type_b;
    p->out_dtype = out_dtype;
    p->layout_a = layout_a;
    p->layout_b = layout_b;
    p->scale_a = scale_a;
    p->scale_b = scale_b;
    p->device = dev;
    p->num_sms = num_sms;
    p->offline = offline;
    p->opt_form = -1;
    const gemm_status_t st = derive(p);
    if (st != GEMM_OK) {
        delete p;
        return st;
    }
    const int zeros[G_WORDS] = {};
    if (!offline && (cudaMalloc(&p->d_status, sizeof(zeros)) != cudaSuccess || !upload(p->d_status, zeros, sizeof(zeros)))) {
        cudaGetLastError();
        if (p->d_status) cudaFree(p->d_status);
        delete p;
        return GEMM_ERR_CUDA;
    }
    *out = p;
    return GEMM_OK;
}

// Map of a matrix of y rows of x elements.
bool encode(CUtensorMap* m, CUtensorMapDataType type, int size, const void* base, int64_t x, int64_t y, uint32_t box_x, uint32_t box_y,
            CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)x, (cuuint64_t)y};
    const cuuint64_t strides[1] = {(cuuint64_t)x * (cuuint64_t)size};
    const cuuint32_t box[2] = {box_x, box_y};
    const cuuint32_t estr[2] = {1, 1};
    return enc(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool W, bool X>
auto few_of(int rows) -> void (*)(FewParams) {
    return rows <= 8 ? few_kernel<W, X, 1> : rows <= 16 ? few_kernel<W, X, 2> : rows <= 24 ? few_kernel<W, X, 3> : few_kernel<W, X, 4>;
}

gemm_status_t run_few(const gemm_scaled_plan* p, const FewParams& kp, gemm_stream_t stream) {
    const bool w = p->type_b == GEMM_E5M2, x = p->type_a == GEMM_E5M2;
    const dim3 grid((unsigned)cdiv(kp.N, 16), (unsigned)cdiv(kp.M, F_MOST_ROWS));
    auto* fn = w ? (x ? few_of<true, true>(kp.M) : few_of<true, false>(kp.M)) : (x ? few_of<false, true>(kp.M) : few_of<false, false>(kp.M));
    return launch(fn, grid, dim3(32 * F_WARPS), 0, stream, kp);
}

// One operand, as the lanes or the columns side sees it: `rows` of K elements.
struct Side {
    const void* q;
    int64_t rows, K;
    bool mn;
    ScaledScales s;
};

Side side_of(const void* q, const float* s, int64_t rows, int64_t K, bool k_major, int scale) {
    Side o{};
    o.q = q;
    o.rows = rows;
    o.K = K;
    o.mn = !k_major;
    o.s.s = s;
    o.s.rows = (int32_t)rows;
    if (scale == GEMM_SCALE_VECTOR) {
        o.s.row = 1;
        o.s.group = rows;
    } else {
        o.s.shift = 7;
        o.s.row = k_major ? cdiv(K, S_BK) : 1;
        o.s.group = k_major ? 1 : cdiv(rows, S_BK);
    }
    return o;
}

bool encode_side(CUtensorMap* m, const Side& o, uint32_t rows) {
    return o.mn ? encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, o.q, o.rows, o.K, 128, S_BK)
                : encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, o.q, o.K, o.rows, S_BK, rows);
}

}  // namespace

extern "C" {

gemm_status_t gemm_scaled_plan_create(gemm_scaled_plan_t* out, int64_t M, int64_t N, int64_t K,
                                      gemm_fp8_t type_a, gemm_fp8_t type_b, int out_dtype,
                                      gemm_layout_t layout_a, gemm_layout_t layout_b,
                                      gemm_scale_t scale_a, gemm_scale_t scale_b) {
    return make_plan(out, M, N, K, type_a, type_b, out_dtype, layout_a, layout_b, scale_a, scale_b, false, 0);
}

gemm_status_t gemm_scaled_plan_create_offline(gemm_scaled_plan_t* out, int64_t M, int64_t N, int64_t K,
                                              gemm_fp8_t type_a, gemm_fp8_t type_b, int out_dtype,
                                              gemm_layout_t layout_a, gemm_layout_t layout_b,
                                              gemm_scale_t scale_a, gemm_scale_t scale_b, int num_sms) {
    return make_plan(out, M, N, K, type_a, type_b, out_dtype, layout_a, layout_b, scale_a, scale_b, true, num_sms);
}

gemm_status_t gemm_scaled_plan_set_option(gemm_scaled_plan_t p, int key, int64_t value) {
    if (!p) return GEMM_ERR_INVALID_ARG;
    if (key == GEMM_SCALED_OPT_INJECT_GIVE_UP) {
        if (value < -1 || value >= p->shape.units) return GEMM_ERR_UNSUPPORTED;
        if (p->offline) return GEMM_ERR_NO_DEVICE;
        DeviceGuard guard(p->device);
        const int word = (int)value + 1;
        return guard.ok && upload(p->d_status + G_WORD_GIVE_UP, &word, sizeof(int)) ? GEMM_OK : GEMM_ERR_CUDA;
    }
    const int saved[2] = {p->opt_ctas, p->opt_form};
    if (key == GEMM_SCALED_OPT_CTAS) {
        if (value < 0 || value > 2) return GEMM_ERR_UNSUPPORTED;
        p->opt_ctas = (int)value;
    } else if (key == GEMM_SCALED_OPT_FORM) {
        if (value < -1 || value > GEMM_SCALED_FEW) return GEMM_ERR_UNSUPPORTED;
        p->opt_form = (int)value;
    } else {
        return GEMM_ERR_INVALID_ARG;
    }
    gemm_status_t st = GEMM_ERR_CUDA;
    if (p->offline) {
        st = derive(p);
    } else {
        DeviceGuard guard(p->device);
        if (guard.ok) st = derive(p);
    }
    if (st != GEMM_OK) {
        p->opt_ctas = saved[0];
        p->opt_form = saved[1];
        derive(p);
    }
    return st;
}

gemm_status_t gemm_scaled_plan_get_info(gemm_scaled_plan_t p, int key, int64_t* value) {
    if (!p || !value) return GEMM_ERR_INVALID_ARG;
    switch (key) {
        case GEMM_SCALED_INFO_CTAS: *value = p->ctas; break;
        case GEMM_SCALED_INFO_FORM: *value = p->form; break;
        case GEMM_SCALED_INFO_UNITS: *value = p->shape.units; break;
        case GEMM_SCALED_INFO_TILES: *value = p->shape.tiles; break;
        case GEMM_SCALED_INFO_TILE_WIDTH: *value = p->shape.width; break;
        case GEMM_SCALED_INFO_SHARES: *value = p->form == GEMM_SCALED_FEW ? 1 : p->shape.shares; break;
        default: return GEMM_ERR_INVALID_ARG;
    }
    return GEMM_OK;
}

gemm_status_t gemm_scaled_workspace_size(gemm_scaled_plan_t p, size_t* bytes) {
    if (!p || !bytes) return GEMM_ERR_INVALID_ARG;
    *bytes = p->ws_bytes;
    return GEMM_OK;
}

gemm_status_t gemm_scaled_run(gemm_scaled_plan_t p, const void* A, const float* scales_a,
                              const void* B, const float* scales_b, void* C, void* workspace,
                              gemm_stream_t stream) {
    if (!p) return GEMM_ERR_INVALID_ARG;
    if (p->offline) return GEMM_ERR_NO_DEVICE;
    if (p->M == 0 || p->N == 0) return GEMM_OK;  // C is empty
    if (!C || (p->K > 0 && (!A || !B || !scales_a || !scales_b))) return GEMM_ERR_INVALID_ARG;
    const int size = p->out_dtype == GEMM_F32 ? 4 : 2;
    if (misaligned(A, 16) || misaligned(B, 16) || misaligned(C, (size_t)size) || misaligned(scales_a, 4) || misaligned(scales_b, 4))
        return GEMM_ERR_UNSUPPORTED;
    if (p->ws_bytes > 0 && (!workspace || misaligned(workspace, 16))) return GEMM_ERR_WORKSPACE;
    DeviceGuard guard(p->device);
    if (!guard.ok) return GEMM_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (p->K == 0)  // empty sums: +0
        return cudaMemsetAsync(C, 0, (size_t)p->M * (size_t)p->N * (size_t)size, st) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
    if (p->form == GEMM_SCALED_FEW) {
        FewParams kp{};
        kp.a = static_cast<const uint8_t*>(A);
        kp.b = static_cast<const uint8_t*>(B);
        kp.sa = side_of(A, scales_a, p->M, p->K, true, p->scale_a).s;
        kp.sb = side_of(B, scales_b, p->N, p->K, true, p->scale_b).s;
        kp.out = C;
        kp.K = p->K;
        kp.N = p->N;
        kp.M = (int32_t)p->M;
        kp.kb = p->shape.kb;
        kp.out_dtype = p->out_dtype;
        return run_few(p, kp, stream);
    }
    if (!prepared(p->ctas, p->turned, p->col_vector, p->device)) return GEMM_ERR_CUDA;

    const Side a = side_of(A, scales_a, p->M, p->K, p->layout_a == GEMM_ROW_MAJOR, p->scale_a);
    const Side b = side_of(B, scales_b, p->N, p->K, p->layout_b == GEMM_COL_MAJOR, p->scale_b);
    const Side &l = p->turned ? b : a, &r = p->turned ? a : b;
    ScaledParams kp{};
    kp.s = p->shape;
    kp.l_total = (int32_t)l.rows;
    kp.l = l.s;
    kp.r = r.s;
    kp.out = C;
    kp.ldc = p->N;
    kp.out_dtype = p->out_dtype;
    kp.boxes = !p->turned && !misaligned(C, 16) && p->N * size % 16 == 0;
    kp.l_mn = l.mn;
    kp.r_mn = r.mn;
    // The maps are encoded for every run: they cost well under a microsecond
    // of host time, and nothing is kept by an operand's address.
    ScaledMaps tm{};
    bool ok = encode_side(&tm.l, l, 128) && encode_side(&tm.r, r, (uint32_t)(p->shape.width / p->ctas));
    if (kp.boxes)
        ok = ok && encode(&tm.c, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, size, C, p->N, p->M,
                          (uint32_t)(64 / size), 32, CU_TENSOR_MAP_SWIZZLE_64B);
    if (!ok) return GEMM_ERR_UNSUPPORTED;
    if (p->ws_bytes > 0) {
        kp.counters = reinterpret_cast<unsigned long long*>(workspace);
        kp.partials = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + p->counter_bytes);
    }
    kp.epoch = next_epoch();
    kp.status = p->d_status;
    const int l_e5m2 = (p->turned ? p->type_b : p->type_a) == GEMM_E5M2, r_e5m2 = (p->turned ? p->type_a : p->type_b) == GEMM_E5M2;
    kp.idesc = idesc_f16(0, l.mn, r.mn, 128 * p->ctas, 0) | ((uint32_t)l_e5m2 << 7) | ((uint32_t)r_e5m2 << 10);
    // a wait may last as long as the longest tile's k-loop
    kp.pipe_limit_ns = 4000000000ull + 2000ull * (uint64_t)p->shape.kb;

    const Kernel k = kernel_of(p->ctas, p->turned, p->col_vector);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p->shape.units * p->ctas), 1, 1);
    cfg.blockDim = dim3(S_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)k.smem;
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
    void* args[2] = {&tm, &kp};
    if (cudaLaunchKernelExC(&cfg, k.fn, args) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

gemm_status_t gemm_scaled_last_status(gemm_scaled_plan_t p, gemm_stream_t stream) {
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
    if (cudaDeviceSynchronize() != cudaSuccess || !upload(p->d_status, words, sizeof(words))) return GEMM_ERR_CUDA;
    ++p->timeouts;
    return GEMM_ERR_TIMEOUT;
}

gemm_status_t gemm_scaled_plan_destroy(gemm_scaled_plan_t p) {
    if (!p) return GEMM_OK;
    if (p->d_status) cudaFree(p->d_status);
    delete p;
    return GEMM_OK;
}

}  // extern "C"
