// Scaled products on the tensor cores: 8-bit floating point in, a scale for each
// 128 summed elements, fp32 accumulation in registers, fp16, bf16 or fp32 out.
//
// Mathematics.  out[l][c] = sum over g of sl(l, g) * sr(c, g) * P_g[l][c], where
// P_g is the product of the 8-bit values over the 128 elements of group g.  The
// tensor cores compute each P_g into tensor memory, from zero; the epilogue warps
// read it and add it, scaled, to sums in registers, while the tensor cores compute
// the next one into another part of tensor memory.  So a k-block is a group, and
// the epilogue runs once a k-block, not once a tile.
//
// Orientation.  L, the operand along the tensor memory's lanes, and R, along its
// columns:
//   straight  L = A, R = B: a lane has a row of C.  The scale of a column operand in
//             blocks is one number for each half of a tile, so an element takes one
//             multiply-add.
//   TURNED    L = B, R = A, for few rows of A: the instruction's N takes any
//             multiple of 16, so that 16 rows cost 16 columns, and 32 lanes store
//             32 neighbours of a row of C.
//
// COLS, how a column's scale is had:
//   0  R in blocks: one number for a half tile.
//   1  a number a column, from shared memory; L's is the same for all lanes of the
//      tile (blocks) and multiplied in there.
//   2  as 1, but L has a number a lane: two operations an element.
//
// PAIR: the two CTAs of a cluster run one tcgen05.mma.cta_group::2 of 256 x 256;
// each CTA keeps its 128 lanes' L and half of R.  Without it, 128 x up to 128 a CTA.
//
// Warp roles (384 threads, one CTA per SM) as in grouped_kernel.cuh: 0 copies, 1
// issues the MMAs, 2 allocates tensor memory, 3 schedules, 4-11 are the epilogue,
// whose two halves have the two halves of a tile's columns.  Split tiles likewise:
// partials in the workspace, the last contributor adds them in ascending k.
//
// Waits inside the CTA are bounded.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "grouped_sched.cuh"
#include "join.cuh"
#include "ptx.cuh"

namespace psm {

constexpr int S_THREADS = 384;
constexpr int S_BK = 128;
constexpr int S_EPI_WARP0 = 4;
constexpr int S_EPI_THREADS = 256;
constexpr int S_QUEUE = 4;
enum : uint32_t { S_BAR_EPI = 1, S_BAR_VOTE = 2 };

template <bool PAIR, bool TURNED, int COLS>
struct ScaledCfg {
    static constexpr int CM = PAIR ? 2 : 1;
    static constexpr int TILE_N = 128 * CM;
    static constexpr int HALF = TILE_N / 2;       // columns of an epilogue half at most
    static constexpr int L_BYTES = 128 * S_BK;
    static constexpr int R_BYTES = 128 * S_BK;    // this CTA's columns
    static constexpr int STAGE_BYTES = L_BYTES + R_BYTES;
    static constexpr int STAGES = COLS == 0 || TURNED ? 6 : 5;
    static constexpr int BUFFERS = 512 / TILE_N;  // products in tensor memory
    static constexpr int BOX_BYTES = TURNED ? 0 : 8 * 4096;              // a staged box a warp
    static constexpr int SCALE_BYTES = COLS == 0 ? 0 : 8 * 2 * HALF * 4; // two k-blocks' a warp
    static constexpr int QUEUE_BYTES = S_QUEUE * 48;
    static constexpr int BAR_BYTES = 320;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + BOX_BYTES + SCALE_BYTES + QUEUE_BYTES + BAR_BYTES + 1024;
    static constexpr int SLOT_FLOATS = 128 * TILE_N;
    static constexpr int BARS = 2 * STAGES + 2 * BUFFERS + 1 + 2 * S_QUEUE;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
    static_assert(BARS * 8 + 32 <= BAR_BYTES, "barrier area");
};

// Scales of one operand: that of row r and k-block g at
// s[(r >> shift) * row + g * group].
struct ScaledScales {
    const float* s;
    int64_t row, group;
    int32_t shift, rows;
};

struct ScaledParams {
    GroupedShape s;               // one group: the columns side
    int32_t l_total;              // extent of the lanes side
    ScaledScales l, r;
    void* out;
    int64_t ldc;                  // elements of a row of C
    int32_t out_dtype;            // 0 f16, 1 bf16, 2 f32
    int32_t boxes;                // straight: C is written by tensor copies
    int32_t l_mn, r_mn;           // operand is MN-major (the summed dimension is strided)
    float* partials;              // a slot a CTA
    unsigned long long* counters; // one a split tile and CTA of the pair
    uint64_t epoch;
    int* status;                  // G_WORD_ words of the plan
    uint32_t idesc;               // without N
    uint64_t pipe_limit_ns;
};

struct ScaledMaps {
    CUtensorMap l, r, c;
};

// ---------------------------------------------------------------- instructions
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void mma_f8_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

// 32 lanes x 16 columns, without the wait.
__device__ __forceinline__ void tmem_ld_x16_async(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Wait for this warp's loads; no use of the registers can be scheduled before it.
__device__ __forceinline__ void tmem_wait_x16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// Two fp32 values in a register pair, and their operations (each rounds to nearest).
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ uint64_t pack_f32x2(uint32_t a, uint32_t b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(a), "r"(b));
    return v;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}

template <int N>
__device__ __forceinline__ void registers_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void registers_fewer() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ uint32_t scaled_pack2(bool bf16, float a, float b) {
    if (bf16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}

// One element to C.
__device__ __forceinline__ void scaled_store(void* out, int dtype, int64_t at, float v) {
    if (dtype == 2) static_cast<float*>(out)[at] = v;
    else if (dtype == 1) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
    else static_cast<__half*>(out)[at] = __float2half_rn(v);
}

// AND of a predicate over the epilogue threads.
__device__ __forceinline__ bool scaled_vote_all(bool v) {
    uint32_t out;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(out)
        : "r"((uint32_t)v), "r"((uint32_t)S_BAR_VOTE), "r"((uint32_t)S_EPI_THREADS)
        : "memory");
    return out != 0;
}

template <bool PAIR, bool TURNED, int COLS>
__global__ void __launch_bounds__(S_THREADS, 1)
    scaled_kernel(const __grid_constant__ ScaledMaps tm, const __grid_constant__ ScaledParams p) {
    using Cf = ScaledCfg<PAIR, TURNED, COLS>;
    static_assert(!TURNED || (!PAIR && COLS > 0), "a turned tile's columns start anywhere");
    constexpr int STAGES = Cf::STAGES, BUFFERS = Cf::BUFFERS, HALF = Cf::HALF;
    constexpr uint16_t PAIR_MASK = 0x3;
    extern __shared__ uint8_t smem_raw[];

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    const uint32_t ring = raw + pad;
    const uint32_t boxes = ring + STAGES * Cf::STAGE_BYTES;
    const uint32_t col_scales = boxes + Cf::BOX_BYTES;
    const uint32_t queue = col_scales + Cf::SCALE_BYTES;
    uint8_t* bar_area = smem_raw + (queue + Cf::QUEUE_BYTES - raw);
    const uint32_t bar_base = smem_addr(bar_area);
    auto full_bar = [&](int s) { return bar_base + 8u * s; };
    auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
    auto tfull_bar = [&](int b) { return bar_base + 8u * (2 * STAGES + b); };
    auto tempty_bar = [&](int b) { return bar_base + 8u * (2 * STAGES + BUFFERS + b); };
    const uint32_t done_bar = bar_base + 8u * (2 * STAGES + 2 * BUFFERS);
    auto qfull_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + 2 * BUFFERS + 1 + s); };
    auto qempty_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + 2 * BUFFERS + 1 + S_QUEUE + s); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_area + 8 * Cf::BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_area + 8 * Cf::BARS + 4);
    volatile int* last_flag = reinterpret_cast<volatile int*>(bar_area + 8 * Cf::BARS + 8);
    int32_t* table = reinterpret_cast<int32_t*>(bar_area + 8 * Cf::BARS + 16);  // offsets, first tiles

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.x / Cf::CM;
    const int rank = PAIR ? (int)cluster_ctarank() : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < BUFFERS; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), Cf::CM * S_EPI_THREADS / 32);
        }
        mbar_init(done_bar, 1);
        // readers of the queue: producer, issuer (pair: the first CTA's) and the epilogue warps
        const int readers = 1 + (!PAIR || rank == 0) + S_EPI_THREADS / 32;
        for (int s = 0; s < S_QUEUE; ++s) {
            mbar_init(qfull_bar(s), 1);
            mbar_init(qempty_bar(s), readers);
        }
        *abort_flag = 0;
        table[0] = table[2] = 0;
        table[1] = p.s.rows;
        table[3] = grouped_tiles(p.s, p.s.rows);
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm.l);
        tma_prefetch_desc(&tm.r);
    }
    if (warp == 2) {
        if constexpr (PAIR) {
            tmem_alloc_pair(smem_addr(tmem_slot), 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_addr(tmem_slot), 512);
            tmem_relinquish();
        }
    }
    tc_fence_before_sync();
    if constexpr (PAIR) cluster_sync_all();
    else __syncthreads();
    tc_fence_after_sync();
    // everything above may overlap the previous kernel in the stream
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    const uint32_t tmem_base = *tmem_slot;

    auto fail_pipe = [&]() {
        *abort_flag = 1;
        atomicCAS(p.status + G_WORD_STATUS, 0, G_STATUS_PIPE_TIMEOUT);
    };

    GroupedWork w{};
    int qslot = 0;
    uint32_t qphase = 0;
    // The next piece of work, for a whole warp; false at the end or after a
    // wait that ran out.
    auto next_work = [&]() {
        const bool got = mbar_wait(qfull_bar(qslot), qphase, p.pipe_limit_ns);
        if (!__all_sync(0xffffffffu, got && *abort_flag == 0)) {
            if (lane == 0) fail_pipe();
            return false;
        }
        const uint32_t at = queue + (uint32_t)qslot * 48u;
        const uint4 a = ld_shared_u4(at), b = ld_shared_u4(at + 16), c = ld_shared_u4(at + 32);
        __syncwarp();
        if (lane == 0) mbar_arrive(qempty_bar(qslot));
        if (++qslot == S_QUEUE) {
            qslot = 0;
            qphase ^= 1u;
        }
        w = GroupedWork{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y,
                        (int)b.z, (int)b.w, (int)c.x, (int)c.y, (int)c.z, (int)c.w};
        return w.item >= 0;
    };

    if (warp < S_EPI_WARP0) {
        if constexpr (PAIR) registers_fewer<72>();
        if (warp == 0) {
            // -------------------------------------------------------- producer
            int stage = 0;
            uint32_t phase = 0;
            uint32_t filled = 0, fill_parity = 0;
            bool ok = true;
            const uint32_t full0_c = PAIR ? mapa_shared(full_bar(0), 0) : 0u;
            while (ok && next_work()) {
                const int l0 = (w.tm * Cf::CM + rank) * 128;
                const int cols = w.width / Cf::CM;  // this CTA's columns
                const int r0 = w.n0 + rank * cols;
                const uint32_t r_bytes = p.r_mn ? (uint32_t)Cf::R_BYTES : (uint32_t)cols * S_BK;
                for (int kb = w.k0; kb < w.k1; ++kb) {
                    if (!__all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1u, p.pipe_limit_ns))) {
                        if (lane == 0) fail_pipe();
                        ok = false;
                        break;
                    }
                    const uint32_t sl = ring + stage * Cf::STAGE_BYTES;
                    const uint32_t sr = sl + Cf::L_BYTES;
                    const uint32_t fb = full_bar(stage), fbc = full0_c + 8u * (uint32_t)stage;
                    auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y) {
                        if constexpr (PAIR) tma_load_2d_pair(dst, map, fbc, x, y, false, 0);
                        else tma_load_2d(dst, map, fb, x, y, false, 0);
                    };
                    if (elect_one()) {
                        const int k = kb * S_BK;
                        if (rank == 0) mbar_arrive_expect_tx(fb, Cf::CM * (Cf::L_BYTES + r_bytes));
                        load(sl, &tm.l, p.l_mn ? l0 : k, p.l_mn ? k : l0);
                        load(sr, &tm.r, p.r_mn ? r0 : k, p.r_mn ? k : r0);
                    }
                    __syncwarp();
                    filled |= 1u << stage;
                    fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // before the CTA (or its peer) exits: every copy has landed, and every
            // MMA that reads this ring has released it
            for (int s = 0; s < STAGES; ++s)
                if (filled & (1u << s)) {
                    if (!PAIR || rank == 0) mbar_wait(full_bar(s), (fill_parity >> s) & 1u, p.pipe_limit_ns);
                    mbar_wait(empty_bar(s), (fill_parity >> s) & 1u, p.pipe_limit_ns);
                }
        } else if (warp == 1) {
            // -------------------------------------------------------- MMA issuer
            if (!PAIR || rank == 0) {
                int stage = 0, buf = 0;
                uint32_t phase = 0, tphase = 0;
                bool ok = true;
                const uint64_t l_desc0 = smem_desc_sw128(ring, p.l_mn ? Cf::L_BYTES : 16, 1024);
                const uint64_t r_desc0 = smem_desc_sw128(ring + Cf::L_BYTES, p.r_mn ? Cf::R_BYTES : 16, 1024);
                // 32 elements of the summed dimension: bytes of a row, or 32 rows of 128 bytes
                const uint64_t l_step = p.l_mn ? (32 * 128) >> 4 : 32 >> 4;
                const uint64_t r_step = p.r_mn ? (32 * 128) >> 4 : 32 >> 4;
                while (ok && next_work()) {
                    const uint32_t idesc = p.idesc | ((uint32_t)(w.width >> 3) << 17);
                    for (int kb = w.k0; kb < w.k1; ++kb) {
                        const bool got = mbar_wait(tempty_bar(buf), tphase ^ 1u, p.pipe_limit_ns) &&
                                         mbar_wait(full_bar(stage), phase, p.pipe_limit_ns) && *abort_flag == 0;
                        if (!__all_sync(0xffffffffu, got)) {
                            if (lane == 0) fail_pipe();
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
                        const uint32_t d_tmem = tmem_base + (uint32_t)(buf * Cf::TILE_N);
                        if (elect_one()) {
                            const uint64_t at = (uint64_t)((uint32_t)(stage * Cf::STAGE_BYTES) >> 4);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                const uint64_t ld = l_desc0 + at + (uint64_t)kk * l_step;
                                const uint64_t rd = r_desc0 + at + (uint64_t)kk * r_step;
                                if constexpr (PAIR) mma_f8_ss_pair(d_tmem, ld, rd, idesc, kk > 0);
                                else mma_f8_ss(d_tmem, ld, rd, idesc, kk > 0);
                            }
                            if constexpr (PAIR) {
                                mma_commit_pair_multicast(empty_bar(stage), PAIR_MASK);
                                mma_commit_pair_multicast(tfull_bar(buf), PAIR_MASK);
                            } else {
                                mma_commit(empty_bar(stage));
                                mma_commit(tfull_bar(buf));
                            }
                        }
                        __syncwarp();
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        if (++buf == BUFFERS) {
                            buf = 0;
                            tphase ^= 1u;
                        }
                    }
                }
                // all MMAs are complete before tensor memory is freed
                __syncwarp();
                if (elect_one()) {
                    if constexpr (PAIR) mma_commit_pair_multicast(done_bar, 0x1);
                    else mma_commit(done_bar);
                }
                __syncwarp();
                mbar_wait(done_bar, 0, p.pipe_limit_ns);
            }
        } else if (warp == 3) {
            // -------------------------------------------------------- scheduler
            const uint64_t tag = grouped_tag(p.epoch, p.status);
            const GroupedTables tab{table, table + 2};
            const int32_t items = table[3];
            const GroupedSplit split = grouped_split(p.s, items, 0);
            bool more = true;
            for (int32_t step = 0; more; ++step) {
                more = grouped_work(p.s, tab, split, unit, step, items, w);
                if (!more) w.item = -1;
                if (!__all_sync(0xffffffffu, mbar_wait(qempty_bar(qslot), qphase ^ 1u, p.pipe_limit_ns))) {
                    if (lane == 0) fail_pipe();
                    break;
                }
                if (lane == 0) {
                    const uint32_t at = queue + (uint32_t)qslot * 48u;
                    st_shared_u4(at, w.item, w.shares, w.group, w.tm);
                    st_shared_u4(at + 16, w.n0, w.width, w.valid, w.r0);
                    st_shared_u4(at + 32, w.r1, w.k0, w.k1, w.kb);
                    mbar_arrive(qfull_bar(qslot));
                    if (more && w.shares > 1 && w.item == unit)  // this unit has the first share
                        grouped_open_counter(p.counters + (size_t)unit * Cf::CM + rank, tag);
                }
                __syncwarp();
                if (++qslot == S_QUEUE) {
                    qslot = 0;
                    qphase ^= 1u;
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        if constexpr (PAIR) registers_more<216>();
        const int q = warp & 3;  // tensor-memory lanes 32q .. 32q + 31
        const int half = (warp - S_EPI_WARP0) >> 2;
        const int et = threadIdx.x - S_EPI_WARP0 * 32;
        const uint64_t tag = grouped_tag(p.epoch, p.status);
        const bool give_up = p.status[G_WORD_GIVE_UP] == unit + 1;
        const uint32_t my_scales = col_scales + (uint32_t)(warp - S_EPI_WARP0) * (2 * HALF * 4);
        const uint32_t my_box = boxes + (uint32_t)(warp - S_EPI_WARP0) * 4096u;
        const uint32_t release0 = PAIR ? mapa_shared(tempty_bar(0), 0) : tempty_bar(0);
        constexpr int PER = HALF / 32;  // column scales a lane fetches
        constexpr int VALUES = COLS == 0 ? 2 : 1 + PER;
        int buf = 0;
        uint32_t tphase = 0;
        while (next_work()) {
            // this half's columns: c0 .. c0 + 16 * chunks - 1 of the tile
            const int half_width = PAIR ? HALF : ((w.width >> 1) + 15) & ~15;
            const int c0 = half * half_width;
            const int chunks = PAIR ? HALF / 16 : max(0, min(w.width - c0, half_width)) >> 4;
            const int l = (w.tm * Cf::CM + rank) * 128 + q * 32 + lane;
            // the scales' addresses; rows and columns past the end read the last one's
            const float* ls = p.l.s + (int64_t)(min(l, p.l.rows - 1) >> p.l.shift) * p.l.row;
            const float* rs[COLS == 0 ? 1 : PER];
            if constexpr (COLS == 0) {
                rs[0] = p.r.s + (int64_t)(min(w.n0 + c0, p.r.rows - 1) >> p.r.shift) * p.r.row;
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    rs[i] = p.r.s + (int64_t)(min(w.n0 + c0 + lane * PER + i, p.r.rows - 1) >> p.r.shift) * p.r.row;
            }
            // fetched two k-blocks ahead
            float now[VALUES], next[VALUES], after[VALUES];
            auto fetch = [&](int kb, float (&v)[VALUES]) {
                const int64_t g = min(kb, w.k1 - 1);
                v[0] = ls[g * p.l.group];
#pragma unroll
                for (int i = 0; i < VALUES - 1; ++i) v[1 + i] = rs[i][g * p.r.group];
            };
            uint64_t acc[HALF / 2];
#pragma unroll
            for (int i = 0; i < HALF / 2; ++i) acc[i] = 0;
            fetch(w.k0, now);
            fetch(w.k0 + 1, next);
            bool ok = !give_up;
#pragma unroll 1
            for (int kb = w.k0; kb < w.k1; ++kb) {
                fetch(kb + 2, after);
                uint64_t factor;
                const uint32_t scales_at = my_scales + (uint32_t)(kb & 1) * (HALF * 4);
                if constexpr (COLS == 0) {
                    const float f = now[0] * now[1];
                    factor = pack_f32x2(f, f);
                } else {
                    factor = pack_f32x2(now[0], now[0]);
                    const float with = COLS == 1 ? now[0] : 1.f;
#pragma unroll
                    for (int i = 0; i < PER; i += 2)
                        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(scales_at + (uint32_t)(lane * PER + i) * 4),
                                     "f"(now[1 + i] * with), "f"(now[2 + i] * with)
                                     : "memory");
                    __syncwarp();
                }
                const bool got = mbar_wait(tfull_bar(buf), tphase, p.pipe_limit_ns) && *abort_flag == 0;
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * Cf::TILE_N + c0);
                // two chunks of 16 columns in turn: one is loaded while the other is added
                uint32_t v[2][16];
                if (chunks > 0) tmem_ld_x16_async(tbase, v[0]);
#pragma unroll
                for (int c = 0; c < HALF / 16; ++c) {
                    if (c < chunks) {
                        tmem_wait_x16(v[c & 1]);
                        if (c + 1 < HALF / 16 && c + 1 < chunks) tmem_ld_x16_async(tbase + (c + 1) * 16, v[(c + 1) & 1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint64_t f[2] = {factor, factor};
                            if constexpr (COLS > 0) {
                                const float4 s = ld_shared_f4(scales_at + (uint32_t)(c * 16 + i * 4) * 4);
                                f[0] = pack_f32x2(s.x, s.y);
                                f[1] = pack_f32x2(s.z, s.w);
                            }
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                uint64_t& a = acc[c * 8 + i * 2 + j];
                                const uint64_t product = pack_f32x2(v[c & 1][i * 4 + j * 2], v[c & 1][i * 4 + j * 2 + 1]);
                                if constexpr (COLS == 2) a = fma_f32x2(mul_f32x2(product, f[j]), factor, a);
                                else a = fma_f32x2(product, f[j], a);
                            }
                        }
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_cluster_fenced(release0 + 8u * (uint32_t)buf);
                    else mbar_arrive(release0 + 8u * (uint32_t)buf);
                }
                if (++buf == BUFFERS) {
                    buf = 0;
                    tphase ^= 1u;
                }
#pragma unroll
                for (int i = 0; i < VALUES; ++i) {
                    now[i] = next[i];
                    next[i] = after[i];
                }
            }
            if (!ok && lane == 0) fail_pipe();
            // (a warp that gives up must not leave the others at a barrier)
            if (!scaled_vote_all(ok)) break;
            if (w.shares > 1) {
                float4* slot = reinterpret_cast<float4*>(p.partials + (size_t)blockIdx.x * Cf::SLOT_FLOATS);
#pragma unroll
                for (int i = 0; i < HALF / 4; ++i)
                    if (i < chunks * 4) {
                        const float2 a = unpack_f32x2(acc[2 * i]), b = unpack_f32x2(acc[2 * i + 1]);
                        st_f4(slot + i * S_EPI_THREADS + et, make_float4(a.x, a.y, b.x, b.y));
                    }
                // the barrier orders the partial's stores before the count, a release
                // and acquire at GPU scope
                named_bar_sync(S_BAR_EPI, S_EPI_THREADS);
                if (et == 0)
                    *last_flag = grouped_count_in(p.counters + (size_t)w.item * Cf::CM + rank, tag, (uint32_t)w.shares);
                named_bar_sync(S_BAR_EPI, S_EPI_THREADS);
                const bool last = *last_flag != 0;
                named_bar_sync(S_BAR_EPI, S_EPI_THREADS);
                if (!last) continue;
#pragma unroll
                for (int i = 0; i < HALF / 2; ++i) acc[i] = 0;
#pragma unroll 1
                for (int x = 0; x < w.shares; ++x) {
                    // share x was run by unit w.item + x
                    const float4* from = reinterpret_cast<const float4*>(
                        p.partials + (size_t)((w.item + x) * Cf::CM + rank) * Cf::SLOT_FLOATS) + et;
                    const uint64_t one = pack_f32x2(1.f, 1.f);
#pragma unroll
                    for (int i = 0; i < HALF / 4; ++i)
                        if (i < chunks * 4) {
                            const float4 y = ld_cg_f4(from + i * S_EPI_THREADS);
                            acc[2 * i] = fma_f32x2(pack_f32x2(y.x, y.y), one, acc[2 * i]);
                            acc[2 * i + 1] = fma_f32x2(pack_f32x2(y.z, y.w), one, acc[2 * i + 1]);
                        }
                }
            }
            // ---- the tile to C
            const int row0 = l - lane;
            if constexpr (TURNED) {
                const int count = min(w.valid - c0, chunks * 16);  // columns with a row of C
                if (l < p.l_total) {
                    const int64_t at = (int64_t)(w.n0 + c0) * p.ldc + l;
#pragma unroll
                    for (int i = 0; i < HALF / 2; ++i) {
                        const float2 x = unpack_f32x2(acc[i]);
                        if (2 * i < count) scaled_store(p.out, p.out_dtype, at + (int64_t)(2 * i) * p.ldc, x.x);
                        if (2 * i + 1 < count) scaled_store(p.out, p.out_dtype, at + (int64_t)(2 * i + 1) * p.ldc, x.y);
                    }
                }
            } else if (p.boxes) {
                // boxes of 32 rows x 128 bytes, 16-byte units swizzled by row
                const uint32_t my_row = my_box + (uint32_t)lane * 128u;
                const int col = w.n0 + c0;
                auto send = [&](int x) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (x < (int)p.ldc && row0 < p.l_total) tma_store_2d(&tm.c, my_box, x, row0);
                        bulk_commit_group();
                    }
                };
                auto free_box = [&]() {
                    if (lane == 0) bulk_wait_group_read_0();
                    __syncwarp();
                };
                if (p.out_dtype == 2) {
#pragma unroll
                    for (int b = 0; b < HALF / 32; ++b) {
                        free_box();
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const float2 x = unpack_f32x2(acc[b * 16 + 2 * u]), y = unpack_f32x2(acc[b * 16 + 2 * u + 1]);
                            st_shared_u4(my_row + (uint32_t)((u ^ (lane & 7)) * 16), __float_as_uint(x.x), __float_as_uint(x.y),
                                         __float_as_uint(y.x), __float_as_uint(y.y));
                        }
                        send(col + b * 32);
                    }
                } else {
                    const bool bf16 = p.out_dtype == 1;
#pragma unroll
                    for (int b = 0; b < HALF / 64; ++b) {
                        free_box();
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            uint32_t o[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 x = unpack_f32x2(acc[b * 32 + 4 * u + i]);
                                o[i] = scaled_pack2(bf16, x.x, x.y);
                            }
                            st_shared_u4(my_row + (uint32_t)((u ^ (lane & 7)) * 16), o[0], o[1], o[2], o[3]);
                        }
                        send(col + b * 64);
                    }
                }
            } else if (l < p.l_total) {
                // rows of C that tensor copies cannot address: element by element
                const int64_t at = (int64_t)l * p.ldc + w.n0 + c0;
                const int64_t count = p.ldc - (w.n0 + c0);
#pragma unroll
                for (int i = 0; i < HALF / 2; ++i) {
                    const float2 x = unpack_f32x2(acc[i]);
                    if (2 * i < count) scaled_store(p.out, p.out_dtype, at + 2 * i, x.x);
                    if (2 * i + 1 < count) scaled_store(p.out, p.out_dtype, at + 2 * i + 1, x.y);
                }
            }
        }
        if (lane == 0) bulk_wait_group_0();  // the copies are complete before the CTA ends
    }

    tc_fence_before_sync();
    __syncwarp();
    if constexpr (PAIR) cluster_sync_all();
    else __syncthreads();
    if (warp == 2) {
        __syncwarp();
        tc_fence_after_sync();
        if constexpr (PAIR) tmem_dealloc_pair(tmem_base, 512);
        else tmem_dealloc(tmem_base, 512);
    }
}

}  // namespace psm
