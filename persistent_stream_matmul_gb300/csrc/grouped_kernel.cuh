// Grouped products on the tensor cores: fp16/bf16 in, fp32 accumulation in
// tensor memory, fp16/bf16 out.
//
// Orientation.  Both kinds compute out[j][m] = sum_k P[m, k] * Q[j, k], with m
// the contiguous dimension of the output, along the tensor memory's lanes, and
// j along its columns:
//   ROWS   P = a group's matrix (m = columns of C), Q = the group's rows of A;
//   INNER  P and Q = the columns of the two row operands, k = the group's rows.
// So the ragged dimension of ROWS is the instruction's N, which takes any
// multiple of 16 (32 for a pair): a group of 300 rows runs as two tiles of 160
// and 140 rows, not as three of 128, and eight rows cost 16.  Rows past a
// group's end that a tile loads (its neighbour's) only reach accumulator
// columns that are not stored.
//
// PAIR: the two CTAs of a cluster run one tcgen05.mma.cta_group::2 of 256 x up
// to 256; each CTA keeps its 128 lanes' P and half of Q.  Without it, 128 x up
// to 128 a CTA.
//
// Warp roles (384 threads, one CTA per SM):
//   warp 0     TMA producer, a ring of STAGES stages of 16 KB of P and up to
//              16 KB of Q (128-byte swizzle), as many rows of Q as the tile has.
//              INNER: a group's last k-block may end inside a 16-row step of
//              the MMA.  Its copies then are cut into boxes of 32, 16, 8 .. 1 rows:
//              the group's rows, then rows past the tensor's end, which read as
//              zeros, up to the next multiple of 16, where the MMA stops.  Zeros in
//              both operands, so that whatever a neighbour's rows hold (NaN,
//              infinity) adds nothing.  Few copies matter: one box a bit of the rows
//              and of the zeros took 984 us where this takes 977 (8 gradients of 14336
//              x 4096 over 16384 rows), and boxes of 3, 5 and 7 rows 990.  All of a block's bytes are counted on its
//              one barrier, so a pair needs no order between one CTA's writes to
//              shared memory and the MMA that the other issues.  (Zeros written by
//              a warp, released at cluster scope: 64 gradients of 2048 x 1536 over
//              512 rows each 157 us against 144.)
//   warp 1     one lane issues the MMAs (pair: the first CTA's, for both).
//   warp 2     allocates tensor memory.
//   warp 3     scheduler: walks this unit's work and hands every piece to the
//              other warps through a queue of G_QUEUE entries in shared memory.
//              With the walk (searches and divisions, ~1000 cycles) repeated
//              in every role, its copies of the code were fetched cold before
//              the first load, and the epilogue paid it between tiles.
//   warps 4-11 epilogue, two halves that take the 32-row chunks of a tile in
//              turn (one half alone takes 730 cycles a chunk, its latencies end
//              to end): accumulator fragments, packed to 16 bits, transposed
//              into shared memory as two 128-byte-swizzled boxes of 32 rows x 64
//              columns.  Tiles of G_BOX_BLOCKS k-blocks or more are written by
//              tensor copies, the others, and the rows before a group's end
//              inside a box, by the lanes, 256 bytes a row.  us, lanes against
//              copies: 16384 rows of 14336 x 4096 1187 / 1178 and their gradient
//              1151 / 1125, where the copies leave the tensor cores more of
//              shared memory; gradients of 64 matrices over 512 rows each (8
//              k-blocks) 143 / 140, over 128 rows 90 / 105, where stores bound.
//
// Split tiles (grouped_sched.cuh): every contributor writes its fp32 partial to
// its workspace slot and counts itself in; the one that comes last adds all
// partials in ascending k and stores.  Nothing waits, and the sum does not
// depend on who comes last.  Joining costs about 3 us, the time of 16 k-blocks
// at the rate of one SM, hence the least share.
//
// Waits inside the CTA are bounded, as in gemm_kernel.cuh.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "grouped_sched.cuh"
#include "join.cuh"
#include "ptx.cuh"

namespace psm {

constexpr int G_THREADS = 384;
constexpr int G_BK = 64;
constexpr int G_EPI_WARP0 = 4;
constexpr int G_EPI_THREADS = 256;
constexpr int G_MAX_GROUPS = 1024;
constexpr int G_QUEUE = 4;
constexpr int G_BOX_BLOCKS = 8;
constexpr uint32_t G_CHUNK = 64 * 128;  // one 64 x 64 MN-major box
enum : uint32_t { G_BAR_EPI = 1, G_BAR_VOTE = 2, G_BAR_HALF = 3 };  // G_BAR_HALF + half

template <bool PAIR>
struct GroupedCfg {
    static constexpr int CM = PAIR ? 2 : 1;
    static constexpr int TILE_N = 128 * CM;
    static constexpr int P_BYTES = 128 * G_BK * 2;
    static constexpr int Q_BYTES = 128 * G_BK * 2;  // this CTA's rows of Q
    static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
    static constexpr int STAGES = 6;
    static constexpr int OUT_BYTES = 32 * 256;    // one staged chunk: 32 rows x 128 columns
    static constexpr int TABLE_BYTES = 2 * (G_MAX_GROUPS + 4) * 4;
    static constexpr int QUEUE_BYTES = G_QUEUE * 48;
    static constexpr int BAR_BYTES = 256;
    static constexpr int TMEM_COLS = 2 * TILE_N;  // two accumulators
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 2 * OUT_BYTES + TABLE_BYTES + QUEUE_BYTES + BAR_BYTES + 1024;
    static constexpr int SLOT_FLOATS = 128 * TILE_N;  // a CTA's partial tile
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
    static_assert((2 * STAGES + 5 + 2 * G_QUEUE) * 8 + 16 <= BAR_BYTES, "barrier area");
};

struct GroupedParams {
    GroupedShape s;
    int32_t m_total;              // extent of the output's contiguous dimension
    int64_t out_group;            // INNER: elements of one output matrix
    void* out;
    const int32_t* offsets;
    float* partials;              // a slot a CTA
    unsigned long long* counters; // one a split tile and CTA of the pair
    uint64_t epoch;               // run number, in the counters' tags, 48 bits
    int* status;                  // G_WORD_ words of the plan
    uint32_t idesc;               // without N
    uint64_t pipe_limit_ns;
};

template <bool OUT_BF16>
__device__ __forceinline__ uint32_t grouped_pack2(float a, float b) {
    if constexpr (OUT_BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    } else {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
}

// One warp: the scheduler's tables from the device offsets, bounded (a value
// out of order or range becomes the nearest one in order and range).  128
// entries at a time, four a lane, the next ones loaded ahead of the scans.
// Returns the k-blocks of all tiles (INNER).
__device__ __forceinline__ int32_t grouped_tables(const GroupedShape& s, const int32_t* offsets, int32_t* off,
                                                  int32_t* first) {
    const int lane = threadIdx.x & 31;
    int32_t v[4], next[4];
    auto load = [&](int base, int32_t (&x)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = base + lane * 4 + i <= s.groups ? offsets[base + lane * 4 + i] : 0;
    };
    load(0, v);
    int32_t top = 0, tiles = 0, blocks = 0, last = 0;  // carried: maximum, sums, and the last entry
    for (int base = 0; base <= s.groups; base += 128) {
        load(base + 128, next);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = max(i ? v[i - 1] : 0, min(v[i], s.rows));
        int32_t m = v[3];
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(0xffffffffu, m, o);
            if (lane >= o) m = max(m, u);
        }
        int32_t before = __shfl_up_sync(0xffffffffu, m, 1);
        before = max(top, lane ? before : 0);
        top = max(top, __shfl_sync(0xffffffffu, m, 31));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = max(v[i], before);
        // entry i closes group i - 1
        int32_t prev = __shfl_up_sync(0xffffffffu, v[3], 1);
        if (lane == 0) prev = last;
        last = __shfl_sync(0xffffffffu, v[3], 31);
        int32_t c[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int g = base + lane * 4 + i;
            if (g > 0 && g <= s.groups) {
                const int32_t n = v[i] - (i ? v[i - 1] : prev);
                const int32_t x = grouped_tiles(s, n);
                sum += x;
                if (s.inner && s.may_split) blocks += x * grouped_k_blocks(s, n);
            }
            c[i] = sum;
        }
        int32_t run = sum;
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t a = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += a;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int g = base + lane * 4 + i;
            if (g <= s.groups) {
                off[g] = v[i];
                first[g] = tiles + run - sum + c[i];
            }
        }
        tiles += __shfl_sync(0xffffffffu, run, 31);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = next[i];
    }
    for (int o = 16; o; o >>= 1) blocks += __shfl_xor_sync(0xffffffffu, blocks, o);
    __syncwarp();
    return blocks;
}

// One warp: `first` in shares instead of tiles.
__device__ __forceinline__ void grouped_split_table(const GroupedShape& s, const int32_t* off, int32_t* first,
                                                    int32_t most) {
    const int lane = threadIdx.x & 31;
    int32_t carry = 0;
    for (int base = 0; base < s.groups; base += 32) {
        const int g = base + lane;
        const int32_t n = g < s.groups ? off[g + 1] - off[g] : 0;
        const int32_t mine = g < s.groups ? grouped_tiles(s, n) * grouped_shares(grouped_k_blocks(s, n), most) : 0;
        int32_t v = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (g < s.groups) first[g] = carry + v - mine;
        carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) first[s.groups] = carry;
    __syncwarp();
}

// AND of a predicate over the epilogue threads.
__device__ __forceinline__ bool grouped_vote_all(bool v) {
    uint32_t out;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(out)
        : "r"((uint32_t)v), "r"((uint32_t)G_BAR_VOTE), "r"((uint32_t)G_EPI_THREADS)
        : "memory");
    return out != 0;
}

// ROWS: p reads the matrices, q[i] boxes of 16 << i rows of A.  INNER: p[i] and
// q[i] read boxes of 1 << i rows.
template <bool INNER>
struct GroupedMaps {
    CUtensorMap p[INNER ? 7 : 1], q[INNER ? 7 : 4], c;
};

// P_MN: P is MN-major (INNER: both operands are).
template <bool PAIR, bool INNER, bool P_MN, bool OUT_BF16>
__global__ void __launch_bounds__(G_THREADS, 1)
    grouped_kernel(const __grid_constant__ GroupedMaps<INNER> tm, const __grid_constant__ GroupedParams p) {
    using Cf = GroupedCfg<PAIR>;
    static_assert(!INNER || P_MN, "INNER reads both operands MN-major");
    constexpr int STAGES = Cf::STAGES;
    constexpr uint16_t PAIR_MASK = 0x3;
    extern __shared__ uint8_t smem_raw[];

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    const uint32_t ring = raw + pad;
    const uint32_t out_stage = ring + STAGES * Cf::STAGE_BYTES;
    uint8_t* tables = smem_raw + pad + STAGES * Cf::STAGE_BYTES + 2 * Cf::OUT_BYTES;
    int32_t* off = reinterpret_cast<int32_t*>(tables);
    int32_t* first = off + G_MAX_GROUPS + 4;
    const uint32_t queue = smem_addr(tables + Cf::TABLE_BYTES);
    uint8_t* bar_area = tables + Cf::TABLE_BYTES + Cf::QUEUE_BYTES;
    const uint32_t bar_base = smem_addr(bar_area);
    auto full_bar = [&](int s) { return bar_base + 8u * s; };
    auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
    auto tfull_bar = [&](int b) { return bar_base + 8u * (2 * STAGES + b); };
    auto tempty_bar = [&](int b) { return bar_base + 8u * (2 * STAGES + 2 + b); };
    const uint32_t done_bar = bar_base + 8u * (2 * STAGES + 4);
    auto qfull_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + 5 + s); };
    auto qempty_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + 5 + G_QUEUE + s); };
    constexpr int BARS = 2 * STAGES + 5 + 2 * G_QUEUE;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_area + 8 * BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_area + 8 * BARS + 4);
    volatile int* last_flag = reinterpret_cast<volatile int*>(bar_area + 8 * BARS + 8);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.x / Cf::CM;
    const int rank = PAIR ? (int)cluster_ctarank() : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), Cf::CM * G_EPI_THREADS / 32);
        }
        mbar_init(done_bar, 1);
        // readers of the queue: producer, issuer (pair: the first CTA's) and the epilogue warps
        const int readers = 1 + (!PAIR || rank == 0) + G_EPI_THREADS / 32;
        for (int s = 0; s < G_QUEUE; ++s) {
            mbar_init(qfull_bar(s), 1);
            mbar_init(qempty_bar(s), readers);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm.p[INNER ? 6 : 0]);
        tma_prefetch_desc(&tm.q[INNER ? 6 : 0]);
    }
    if (warp == 2) {
        if constexpr (PAIR) {
            tmem_alloc_pair(smem_addr(tmem_slot), Cf::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_addr(tmem_slot), Cf::TMEM_COLS);
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
        if (++qslot == G_QUEUE) {
            qslot = 0;
            qphase ^= 1u;
        }
        w = GroupedWork{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y,
                        (int)b.z, (int)b.w, (int)c.x, (int)c.y, (int)c.z, (int)c.w};
        return w.item >= 0;
    };
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int stage = 0;
        uint32_t phase = 0;
        uint32_t filled = 0, fill_parity = 0;
        bool ok = true;
        const uint32_t full0_c = PAIR ? mapa_shared(full_bar(0), 0) : 0u;
        while (ok && next_work()) {
            const int m0 = (w.tm * Cf::CM + rank) * 128;
            const int rows_q = w.width / Cf::CM;  // this CTA's rows of Q
            const int q0 = w.n0 + rank * rows_q;
            // ROWS: the smallest box that holds them (a box a bit of their number,
            // which reads fewer rows in more copies, measured the same)
            const int box = rows_q <= 16 ? 0 : rows_q <= 32 ? 1 : rows_q <= 64 ? 2 : 3;
            const uint32_t q_bytes = (16u << box) * 128u;
            for (int kb = w.k0; kb < w.k1; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1u, p.pipe_limit_ns))) {
                    if (lane == 0) fail_pipe();
                    ok = false;
                    break;
                }
                const uint32_t sp = ring + stage * Cf::STAGE_BYTES;
                const uint32_t sq = sp + Cf::P_BYTES;
                const uint32_t fb = full_bar(stage), fbc = full0_c + 8u * (uint32_t)stage;
                auto load_2d = [&](uint32_t dst, const CUtensorMap* map, int x, int y) {
                    if constexpr (PAIR) tma_load_2d_pair(dst, map, fbc, x, y, false, 0);
                    else tma_load_2d(dst, map, fb, x, y, false, 0);
                };
                // INNER: rows of the group in this block, and up to the next step of 16
                const int k_inner = w.r0 + kb * G_BK, rows = min(G_BK, w.r1 - k_inner), zeros = -rows & 15;
                if (INNER && zeros) {
                    // A lane a copy: four boxes of 64 columns (two of P, two of Q) by four
                    // pieces.  The rows: the largest power of two from their first and
                    // again up to their last (where the two meet they write the same
                    // bytes).  The zeros: likewise where the block ends with them, else 8
                    // or 16 rows, as no MMA reads past the step.
                    const bool ends = rows > 48;
                    const int rb = 31 - __clz(rows), zb = ends ? 31 - __clz(zeros) : zeros > 8 ? 4 : 3;
                    const bool r2 = rows != 1 << rb, z2 = ends && zeros != 1 << zb;
                    if (elect_one() && rank == 0)
                        mbar_arrive_expect_tx(fb, Cf::CM * 4 * 128 * ((1 << rb << r2) + (1 << zb << z2)));
                    const int box64 = lane & 3, piece = lane >> 2;
                    if (piece == 0 || piece == 2 || (piece == 1 && r2) || (piece == 3 && z2)) {
                        const int bit = piece < 2 ? rb : zb;
                        const int at = piece == 0 ? 0 : piece == 1 ? rows - (1 << rb) : piece == 2 ? rows : rows + zeros - (1 << zb);
                        load_2d(sp + box64 * G_CHUNK + at * 128, box64 < 2 ? &tm.p[bit] : &tm.q[bit],
                                (box64 < 2 ? m0 : q0) + 64 * (box64 & 1), piece < 2 ? k_inner + at : p.s.rows);
                    }
                } else if (elect_one()) {
                    if constexpr (INNER) {
                        if (rank == 0) mbar_arrive_expect_tx(fb, Cf::CM * Cf::STAGE_BYTES);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            load_2d(sp + c * G_CHUNK, &tm.p[6], m0 + 64 * c, k_inner);
                            load_2d(sq + c * G_CHUNK, &tm.q[6], q0 + 64 * c, k_inner);
                        }
                    } else {
                        const int k = kb * G_BK;
                        auto load_3d = [&](uint32_t dst, int x, int y) {
                            if constexpr (PAIR) tma_load_3d_pair(dst, &tm.p[0], fbc, x, y, w.group);
                            else tma_load_3d(dst, &tm.p[0], fb, x, y, w.group);
                        };
                        if (rank == 0) mbar_arrive_expect_tx(fb, Cf::CM * (Cf::P_BYTES + q_bytes));
                        if constexpr (P_MN) {
                            load_3d(sp, m0, k);
                            load_3d(sp + G_CHUNK, m0 + 64, k);
                        } else {
                            load_3d(sp, k, m0);
                        }
                        load_2d(sq, &tm.q[box], k, q0);
                    }
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
        // ------------------------------------------------------------ MMA issuer
        if (!PAIR || rank == 0) {
            int stage = 0;
            uint32_t phase = 0, iter = 0;
            bool ok = true;
            const uint64_t p_desc0 = smem_desc_sw128(ring, P_MN ? G_CHUNK : 16, 1024);
            const uint64_t q_desc0 = smem_desc_sw128(ring + Cf::P_BYTES, INNER ? G_CHUNK : 16, 1024);
            constexpr uint64_t p_step = P_MN ? (16 * 128) >> 4 : 32 >> 4;
            constexpr uint64_t q_step = INNER ? (16 * 128) >> 4 : 32 >> 4;
            while (ok && next_work()) {
                if (w.k1 <= w.k0) continue;  // an empty group: the epilogue writes zeros
                const int buf = iter & 1;
                if (!__all_sync(0xffffffffu,
                                mbar_wait(tempty_bar(buf), ((iter >> 1) & 1u) ^ 1u, p.pipe_limit_ns))) {
                    if (lane == 0) fail_pipe();
                    break;
                }
                if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
                tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + (uint32_t)(buf * Cf::TILE_N);
                const uint32_t idesc = p.idesc | ((uint32_t)(w.width >> 3) << 17);
                for (int kb = w.k0; kb < w.k1; ++kb) {
                    if (!__all_sync(0xffffffffu, mbar_wait(full_bar(stage), phase, p.pipe_limit_ns))) {
                        if (lane == 0) fail_pipe();
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const bool leader = elect_one();
                    const uint64_t at = (uint64_t)((uint32_t)(stage * Cf::STAGE_BYTES) >> 4);
                    // k-steps of 16 with rows in them (INNER: a group's last block may have fewer)
                    const int steps = INNER ? min(4, (w.r1 - w.r0 - kb * G_BK + 15) / 16) : 4;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t pd = p_desc0 + at + (uint64_t)kk * p_step;
                        const uint64_t qd = q_desc0 + at + (uint64_t)kk * q_step;
                        const uint32_t acc = (kb > w.k0 || kk > 0) ? 1u : 0u;
                        if (leader && kk < steps) {
                            if constexpr (PAIR) mma_f16_ss_pair(d_tmem, pd, qd, idesc, acc);
                            else mma_f16_ss(d_tmem, pd, qd, idesc, acc);
                        }
                    }
                    if (leader) {
                        if constexpr (PAIR) mma_commit_pair_multicast(empty_bar(stage), PAIR_MASK);
                        else mma_commit(empty_bar(stage));
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                if (elect_one()) {
                    if constexpr (PAIR) mma_commit_pair_multicast(tfull_bar(buf), PAIR_MASK);
                    else mma_commit(tfull_bar(buf));
                }
                __syncwarp();
                ++iter;
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
        // ------------------------------------------------------------ scheduler
        const uint64_t tag = grouped_tag(p.epoch, p.status);
        const int32_t blocks = grouped_tables(p.s, p.offsets, off, first);
        const GroupedTables tab{off, first};
        const int32_t tiles = first[p.s.groups];
        const GroupedSplit split = grouped_split(p.s, tiles, blocks);
        if (INNER && split.most > 0) grouped_split_table(p.s, off, first, split.most);
        const int32_t items = first[p.s.groups];
        bool more = true;
        for (int32_t step = 0; more; ++step) {
            more = grouped_work(p.s, tab, split, unit, step, items, w);
            if (!more) {
                w.item = -1;
                w.r0 = off[0];  // the end carries the rows that belong to a group
                w.r1 = off[p.s.groups];
            }
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
            if (++qslot == G_QUEUE) {
                qslot = 0;
                qphase ^= 1u;
            }
        }
    } else if (warp >= G_EPI_WARP0) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;  // tensor-memory lanes 32q .. 32q + 31
        const int half = (warp - G_EPI_WARP0) >> 2;
        const int et = (threadIdx.x - G_EPI_WARP0 * 32) & 127;  // thread of its half
        const bool lead = threadIdx.x == G_EPI_WARP0 * 32;
        const uint64_t tag = grouped_tag(p.epoch, p.status);
        const bool give_up = p.status[G_WORD_GIVE_UP] == unit + 1;
        uint32_t iter = 0;
        int32_t used0 = 0, used1 = p.s.rows;  // the rows of the groups, from the end of the queue
        auto barrier = [&]() { named_bar_sync(G_BAR_EPI, G_EPI_THREADS); };
        const uint32_t stage_base = out_stage + half * Cf::OUT_BYTES;
        const int read_row = et >> 4, read_unit = et & 15;
        // rows 32c .. 32c + 31 of the tile, from fragments, to the output
        auto store_chunk = [&](const float (&v)[32], int c) {
            if (et == 0) bulk_wait_group_read_0();  // this thread issues the half's copies
            named_bar_sync(G_BAR_HALF + half, 128);  // the last chunk has been read
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = j * 8 + (lane & 7);
                const int u = ((q & 1) * 4 + (lane >> 3)) ^ (row & 7);
                stmatrix_x4_trans(stage_base + (q >> 1) * 4096 + row * 128 + u * 16, grouped_pack2<OUT_BF16>(v[8 * j], v[8 * j + 1]),
                                  grouped_pack2<OUT_BF16>(v[8 * j + 2], v[8 * j + 3]),
                                  grouped_pack2<OUT_BF16>(v[8 * j + 4], v[8 * j + 5]),
                                  grouped_pack2<OUT_BF16>(v[8 * j + 6], v[8 * j + 7]));
            }
            const int col0 = (w.tm * Cf::CM + rank) * 128;
            const bool box = w.kb >= G_BOX_BLOCKS && (INNER || 32 * c + 32 <= w.valid);
            if (box) fence_proxy_async_smem();
            named_bar_sync(G_BAR_HALF + half, 128);
            if (box) {
                if (et == 0) {
                    if (col0 < p.m_total) tma_store_3d(&tm.c, stage_base, col0, w.n0 + 32 * c, INNER ? w.group : 0);
                    if (col0 + 64 < p.m_total) tma_store_3d(&tm.c, stage_base + 4096, col0 + 64, w.n0 + 32 * c, INNER ? w.group : 0);
                    bulk_commit_group();
                }
                return;
            }
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = ld_shared_u4(stage_base + (read_unit >> 3) * 4096 + (read_row + 8 * i) * 128 + (((read_unit & 7) ^ read_row) * 16));
            const int col = col0 + read_unit * 8, row = 32 * c + read_row;
            uint8_t* dst = reinterpret_cast<uint8_t*>(p.out) +
                           2 * ((INNER ? (int64_t)w.group * p.out_group : 0) +
                                (int64_t)(w.n0 + row) * p.m_total + col);
            const int64_t step = (int64_t)p.m_total * 16;  // bytes of 8 rows
            if (col < p.m_total)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (row + 8 * i < w.valid) st_u4(dst + i * step, x[i].x, x[i].y, x[i].z, x[i].w);
        };
        while (true) {
            const bool more = next_work();
            const bool empty = w.k1 <= w.k0;
            const bool split = w.shares > 1;
            const int buf = iter & 1;
            const int chunks = (w.valid + 31) / 32;
            const bool got = more && (empty || (mbar_wait(tfull_bar(buf), (iter >> 1) & 1u, p.pipe_limit_ns) &&
                                                *abort_flag == 0)) && !give_up;
            if (more && !got && lane == 0) fail_pipe();
            // (a warp that gives up must not leave the others at a barrier)
            if (!grouped_vote_all(got)) {
                if (w.item < 0) {
                    used0 = w.r0;
                    used1 = w.r1;
                }
                break;
            }
            if (!empty) {
                tc_fence_after_sync();
            }
            const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * Cf::TILE_N);
            float4* slot = reinterpret_cast<float4*>(p.partials + (size_t)blockIdx.x * Cf::SLOT_FLOATS);
#pragma unroll 1
            for (int c = half; c < chunks; c += 2) {
                uint32_t r[32];
                float v[32];
                if (empty) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.f;
                } else {
                    __syncwarp();
                    tmem_ld_fragments_x4(tbase + c * 32, r);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                }
                if (split) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        st_f4(slot + (c * 8 + i) * 128 + et,
                              make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
                } else {
                    store_chunk(v, c);
                }
            }
            if (!empty) {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_cluster_fenced(mapa_shared(tempty_bar(buf), 0));
                    else mbar_arrive(tempty_bar(buf));
                }
                ++iter;
            }
            if (split) {
                // the barrier orders the partial's stores before the lead's
                // count, a release and acquire at GPU scope
                barrier();
                if (lead)
                    *last_flag = grouped_count_in(p.counters + (size_t)w.item * Cf::CM + rank, tag,
                                                  (uint32_t)w.shares);
                barrier();
                const bool last = *last_flag != 0;
                barrier();
                if (last) {
#pragma unroll 1
                    for (int c = half; c < chunks; c += 2) {
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0.f;
                        // two contributors' loads are in flight together
#pragma unroll 1
                        for (int x = 0; x < w.shares; x += 2) {
                            float4 y[2][8];
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (x + h < w.shares) {
                                    // share x was run by unit w.item + x
                                    const float4* from =
                                        reinterpret_cast<const float4*>(
                                            p.partials + (size_t)((w.item + x + h) * Cf::CM + rank) * Cf::SLOT_FLOATS) +
                                        c * 8 * 128 + et;
#pragma unroll
                                    for (int i = 0; i < 8; ++i) y[h][i] = ld_cg_f4(from + i * 128);
                                }
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (x + h < w.shares)
#pragma unroll
                                    for (int i = 0; i < 8; ++i) {
                                        v[4 * i] += y[h][i].x;
                                        v[4 * i + 1] += y[h][i].y;
                                        v[4 * i + 2] += y[h][i].z;
                                        v[4 * i + 3] += y[h][i].w;
                                    }
                        }
                        store_chunk(v, c);
                    }
                }
            }
        }
        if (et == 0) bulk_wait_group_0();  // the copies are complete before the CTA ends
        if constexpr (!INNER) {
            // the unused rows, before the first group and after the last: +0, 16 bytes a thread
            const int64_t head = (int64_t)used0 * p.m_total / 8, used = (int64_t)(used1 - used0) * p.m_total / 8;
            const int64_t end = (int64_t)p.s.rows * p.m_total / 8 - used;
            for (int64_t i = (int64_t)blockIdx.x * G_EPI_THREADS + (threadIdx.x - G_EPI_WARP0 * 32); i < end;
                 i += (int64_t)gridDim.x * G_EPI_THREADS)
                st_u4(reinterpret_cast<uint8_t*>(p.out) + (i < head ? i : i + used) * 16, 0, 0, 0, 0);
        }
    }

    tc_fence_before_sync();
    __syncwarp();
    if constexpr (PAIR) cluster_sync_all();
    else __syncthreads();
    if (warp == 2) {
        __syncwarp();
        tc_fence_after_sync();
        if constexpr (PAIR) tmem_dealloc_pair(tmem_base, Cf::TMEM_COLS);
        else tmem_dealloc(tmem_base, Cf::TMEM_COLS);
    }
}

}  // namespace psm
