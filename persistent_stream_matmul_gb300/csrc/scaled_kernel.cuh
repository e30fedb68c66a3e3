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
// COL_VECTOR: a scale a column (two operations an element) instead of one for 128 of
// them (one operation, by the product with the lane's).
//
// PAIR: the two CTAs of a cluster run tcgen05.mma.cta_group::2 on a tile of 256 x 256;
// each CTA keeps its 128 lanes' L and half of R.  A k-block is two products of 256 x
// 128, one for each half of the epilogue, with their own buffers and barriers, so that
// the halves run out of step: what one waits for is hidden by the other.  A pair's
// product has 64 columns of each CTA's half of R, so half h has the tile's columns
// 64h .. 64h + 63 and 128 + 64h .. 128 + 64h + 63.
// Without PAIR, 128 x up to 128 a CTA, one product a k-block for both halves.
//
// Warp roles (384 threads, one CTA per SM) as in grouped_kernel.cuh: 0 copies, 1
// issues the MMAs, 2 allocates tensor memory and then copies the scales of the k-blocks
// ahead into a ring of their own, 3 schedules, 4-11 are the epilogue,
// whose two halves have the two halves of a tile's columns.  Split tiles likewise:
// partials in the workspace, the last contributor adds them in ascending k.
//
// What bounds it.  Large products: the epilogue's chain at every k-block (barrier, two
// loads of some 100 cycles, additions), 840 cycles where the tensor cores need 512 and the
// operands' way through shared memory 640: 8192 x 14336 x 4096 takes 342 to 402 us (2.4 to 2.8
// PFLOP/s), with a scale a column 440 to 483 for as many products (14336 x 4096 x 8192). Small
// ones: 2 us to the first copy, and 3 to join split tiles: 96 x 4096 x 14336 takes 20 us,
// 2.9 TB/s.
//
// Waits inside the CTA are bounded.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "join.cuh"
#include "ptx.cuh"

namespace psm {

constexpr int S_EPI_WARPS = 8;
constexpr int S_THREADS = 128 + 32 * S_EPI_WARPS;
constexpr int S_BK = 128;
constexpr int S_EPI_WARP0 = 4;
constexpr int S_EPI_THREADS = 32 * S_EPI_WARPS;
constexpr int S_QUEUE = 4;
// k-blocks of a unit that are brought into L2 ahead (us with 0, 4, 16: 96 x 4096 x 14336 21.2 /
// 20.8 / 21.1, 24 x 4096 x 4096 11.7 / 11.2 / 11.2, 128 x 14336 x 4096 21.2 / 21.4 / 22.3)
constexpr int S_PREFETCH = 4;
constexpr int S_SLOTS = 2;       // of scales, GROUPS k-blocks each
constexpr int S_COL_SCALES = 128 * 4;  // a k-block's: the lanes' scales, then the columns'
constexpr int S_CHUNK = 16;  // columns that a turned tile's half is cut into
// Registers a thread of the pair kernel: at launch (the most that 384 threads can have), and
// in the epilogue, whose eight warps take from the other four what they have more.
constexpr int S_REGS = 168, S_EPI_REGS = 216, S_OTHER_REGS = 3 * S_REGS - 2 * S_EPI_REGS;
enum : uint32_t { S_BAR_EPI = 1, S_BAR_VOTE = 2 };

template <bool PAIR, bool TURNED, bool COL_VECTOR>
struct ScaledCfg {
    static constexpr int CM = PAIR ? 2 : 1;
    static constexpr int TILE_N = 128 * CM;
    static constexpr int PART = TILE_N * 4 / S_EPI_WARPS;  // columns of an epilogue warp at most
    static constexpr int L_BYTES = 128 * S_BK;
    static constexpr int R_BYTES = 128 * S_BK;    // this CTA's columns
    static constexpr int STAGE_BYTES = L_BYTES + R_BYTES;
    // us with 3, 4, 5: pairs, 8192 x 14336 x 4096 365 / 349 / 353, its gradient 455 / 451 /
    // 473; single CTAs, 96 x 4096 x 14336 22.5 / 21.2 / 20.8
    static constexpr int STAGES = PAIR ? 4 : TURNED ? 6 : 5;
    static constexpr int GROUPS = 8;               // k-blocks of a slot of scales
    // staged boxes of a warp, 32 rows x 64 bytes: a ring, of which all but one may still be read
    // when the next is written.  A tile has a whole number of rounds, so it starts with the
    // first.  (us with 2, and with 3 and the ring's place carried on: 8192 x 14336 x 4096 362 / 370,
    // 8192 x 8192 x 128 34.8 / 37.2.)
    static constexpr int BOXES = TURNED ? 0 : 2;
    static constexpr int PRODUCTS = CM;           // products a k-block
    static constexpr int BUFFERS = 4 / PRODUCTS;  // of each, 128 columns of tensor memory
    static constexpr int SCALE_BYTES = S_COL_SCALES + (COL_VECTOR ? TILE_N * 4 : 16);  // of a k-block
    static constexpr int SLOT_BYTES = GROUPS * SCALE_BYTES;
    static constexpr int QUEUE_BYTES = S_QUEUE * 32;
    static constexpr int BAR_BYTES = 384;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + S_EPI_WARPS * BOXES * 2048 + S_SLOTS * SLOT_BYTES + QUEUE_BYTES + BAR_BYTES + 1024;
    static constexpr int SLOT_FLOATS = 128 * TILE_N;
    static constexpr int BARS = 2 * STAGES + 8 + 1 + 2 * S_QUEUE + 2 * S_SLOTS;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
    static_assert(PART / 32 % (BOXES ? BOXES : 1) == 0, "boxes of a tile of 16 bits; 32 bits have twice as many");
    static_assert(BARS * 8 + 32 <= BAR_BYTES, "barrier area");
};

// Tiles and who runs them.  Tiles that do not fill a round of the units (all of them
// when there are fewer than units) run first, the k-blocks of each cut into near-equal
// shares, one a unit at most; then every unit takes whole tiles in turn.  The plan has
// worked out what does not depend on the unit: the first copy starts some 1000 cycles
// after the launch instead of 4000 with the general scheduler of the grouped products.
struct ScaledShape {
    int32_t tiles, tiles_l;       // all tiles; along the lanes side
    int32_t cols, side, width;    // extent of the columns side, tiles along it, and their columns
    int32_t band;                 // tiles along the columns side that are visited before the next lanes tile
    int32_t kb, units;
    int32_t split, shares;        // the first tiles are cut into so many shares
};

struct ScaledWork {
    int32_t item;                 // the unit of the first share; -1: the end
    int32_t shares, tm, n0;       // tile along the lanes; first column
    int32_t valid, k0, k1;        // columns of C; k-blocks
};

// The unit's work number `step`; false past its last.
__device__ __forceinline__ bool scaled_work(const ScaledShape& s, int32_t unit, int32_t step, ScaledWork& w) {
    const bool has = unit < s.split * s.shares;
    uint32_t tile;
    w.shares = 1;
    w.item = unit;
    w.k0 = 0;
    w.k1 = s.kb;
    if (has && step == 0) {
        const int32_t t = unit / s.shares, share = unit - t * s.shares;
        tile = (uint32_t)t;
        w.shares = s.shares;
        w.item = unit - share;
        w.k0 = (int32_t)((int64_t)s.kb * share / s.shares);
        w.k1 = (int32_t)((int64_t)s.kb * (share + 1) / s.shares);
    } else {
        tile = (uint32_t)s.split + (uint32_t)unit + (uint32_t)(step - has) * (uint32_t)s.units;
    }
    if (tile >= (uint32_t)s.tiles) return false;
    const uint32_t in_band = (uint32_t)s.band * (uint32_t)s.tiles_l;
    const uint32_t b = s.band == s.side ? 0u : tile / in_band;
    const uint32_t local = tile - b * in_band;
    const uint32_t first = b * (uint32_t)s.band, wide = min((uint32_t)s.side - first, (uint32_t)s.band);
    w.tm = (int32_t)(wide == 1 ? local : local / wide);
    w.n0 = (int32_t)(first + local - (uint32_t)w.tm * wide) * s.width;
    w.valid = min(s.cols - w.n0, s.width);
    return true;
}

// Scales of one operand: that of row r and k-block g at
// s[(r >> shift) * row + g * group].
struct ScaledScales {
    const float* s;
    int64_t row, group;
    int32_t shift, rows;
};

struct ScaledParams {
    ScaledShape s;
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

// 32 lanes x as many columns as there are registers: the load, and the wait for this
// warp's loads, before which no use of the registers can be scheduled.
__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[64]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]),
                   "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]), "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]),
                   "+r"(r[40]), "+r"(r[41]), "+r"(r[42]), "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]),
                   "+r"(r[48]), "+r"(r[49]), "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]),
                   "+r"(r[56]), "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63]));
}

// Four bytes global -> shared, asynchronously; and an arrival on a barrier (counted in
// its expected ones) when all of this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_4(uint32_t dst_smem, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst_smem), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float ld_shared_f1(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Wait until at most N of this thread's bulk groups have not finished reading their
// shared-memory source.
template <int N>
__device__ __forceinline__ void bulk_wait_group_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// mbar_wait that also gives up once `stop` is set.
__device__ __forceinline__ bool mbar_wait_unless(uint32_t bar, uint32_t parity, uint64_t limit_ns, const volatile int* stop) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*stop != 0 || globaltimer_ns() - t0 > limit_ns) return false;
    }
}

// Whether the phase with the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// Arrivals by one lane without a branch, where the warp has run into them together.
__device__ __forceinline__ void mbar_arrive_if(bool one, uint32_t bar) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%1];\n\t}" ::"r"((uint32_t)one), "r"(bar) : "memory");
}
// (As mbar_arrive_cluster_fenced.)
__device__ __forceinline__ void mbar_arrive_cluster_if(bool one, uint32_t bar) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p mbarrier.arrive.shared::cluster.b64 _, [%1];\n\t}" ::"r"((uint32_t)one), "r"(bar) : "memory");
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

// a[0 .. 3] += v * f (COL_VECTOR: v * f * factor), two at a time: twice as fast as one by
// one where the registers' moves count (8192 x 14336 x 4096 390 us against 435).
template <bool COL_VECTOR>
__device__ __forceinline__ void scaled_add4(float* a, const uint32_t* v, float4 f, float factor) {
    uint64_t v0 = pack_f32x2(v[0], v[1]), v1 = pack_f32x2(v[2], v[3]);
    uint64_t f0 = pack_f32x2(f.x, f.y), f1 = pack_f32x2(f.z, f.w);
    if constexpr (COL_VECTOR) {
        v0 = mul_f32x2(v0, f0);
        v1 = mul_f32x2(v1, f1);
        f0 = f1 = pack_f32x2(factor, factor);
    }
    const float2 x = unpack_f32x2(fma_f32x2(v0, f0, pack_f32x2(a[0], a[1])));
    const float2 y = unpack_f32x2(fma_f32x2(v1, f1, pack_f32x2(a[2], a[3])));
    a[0] = x.x;
    a[1] = x.y;
    a[2] = y.x;
    a[3] = y.y;
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

template <bool PAIR, bool TURNED, bool COL_VECTOR>
__global__ void __launch_bounds__(S_THREADS, 1)
    scaled_kernel(const __grid_constant__ ScaledMaps tm, const __grid_constant__ ScaledParams p) {
    using Cf = ScaledCfg<PAIR, TURNED, COL_VECTOR>;
    static_assert(!TURNED || (!PAIR && COL_VECTOR), "a turned tile's columns start anywhere");
    constexpr int STAGES = Cf::STAGES, BUFFERS = Cf::BUFFERS, PART = Cf::PART;
    constexpr uint16_t PAIR_MASK = 0x3;
    extern __shared__ uint8_t smem_raw[];

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    const uint32_t ring = raw + pad;
    const uint32_t boxes = ring + STAGES * Cf::STAGE_BYTES;
    const uint32_t slots = boxes + S_EPI_WARPS * Cf::BOXES * 2048;
    const uint32_t queue = slots + S_SLOTS * Cf::SLOT_BYTES;
    uint8_t* bar_area = smem_raw + (queue + Cf::QUEUE_BYTES - raw);
    const uint32_t bar_base = smem_addr(bar_area);
    auto full_bar = [&](int s) { return bar_base + 8u * s; };
    auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
    // buffer b of product h is number h * BUFFERS + b of the four
    auto tfull_bar = [&](int b) { return bar_base + 8u * (2 * STAGES + b); };
    auto tempty_bar = [&](int b) { return bar_base + 8u * (2 * STAGES + 4 + b); };
    const uint32_t done_bar = bar_base + 8u * (2 * STAGES + 8);
    auto qfull_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + 9 + s); };
    auto qempty_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + 9 + S_QUEUE + s); };
    auto sfull_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + 9 + 2 * S_QUEUE + s); };
    auto sempty_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + 9 + 2 * S_QUEUE + S_SLOTS + s); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_area + 8 * Cf::BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_area + 8 * Cf::BARS + 4);
    volatile int* last_flag = reinterpret_cast<volatile int*>(bar_area + 8 * Cf::BARS + 8);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.x / Cf::CM;
    const int rank = PAIR ? (int)cluster_ctarank() : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 4; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), Cf::CM / Cf::PRODUCTS * S_EPI_THREADS / 32);
        }
        mbar_init(done_bar, 1);
        for (int s = 0; s < S_SLOTS; ++s) {
            mbar_init(sfull_bar(s), 32);
            mbar_init(sempty_bar(s), S_EPI_THREADS / 32);
        }
        // readers of the queue: producer, copier of the scales, issuer (pair: the first
        // CTA's) and the epilogue warps
        const int readers = 2 + (!PAIR || rank == 0) + S_EPI_THREADS / 32;
        for (int s = 0; s < S_QUEUE; ++s) {
            mbar_init(qfull_bar(s), 1);
            mbar_init(qempty_bar(s), readers);
        }
        *abort_flag = 0;
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
    // Everything above may overlap the previous kernel in the stream, and so may the
    // way of this unit's first boxes of B into L2 (no further: what that kernel may still
    // write there is not read before the wait).
    if (warp == 0) {
        ScaledWork first;
        if (scaled_work(p.s, unit, 0, first) && elect_one()) {
            const int cols = p.s.width / Cf::CM;
            const int at = TURNED ? (first.tm * Cf::CM + rank) * 128 : first.n0 + rank * cols;
            for (int kb = first.k0; kb < min(first.k1, first.k0 + S_PREFETCH); ++kb)
                if (TURNED ? p.l_mn : p.r_mn) tma_prefetch_l2_2d(TURNED ? &tm.l : &tm.r, at, kb * S_BK);
                else tma_prefetch_l2_2d(TURNED ? &tm.l : &tm.r, kb * S_BK, at);
        }
        __syncwarp();
    }
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    const uint32_t tmem_base = *tmem_slot;

    auto fail_pipe = [&]() {
        *abort_flag = 1;
        atomicCAS(p.status + G_WORD_STATUS, 0, G_STATUS_PIPE_TIMEOUT);
    };

    auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait_unless(bar, parity, p.pipe_limit_ns, abort_flag); };
    ScaledWork w{};
    int qslot = 0;
    uint32_t qphase = 0;
    // The next piece of work, for a whole warp; false at the end or after a
    // wait that ran out.
    auto next_work = [&]() {
        const bool got = wait(qfull_bar(qslot), qphase);
        if (!__all_sync(0xffffffffu, got && *abort_flag == 0)) {
            if (lane == 0) fail_pipe();
            return false;
        }
        const uint32_t at = queue + (uint32_t)qslot * 32u;
        const uint4 a = ld_shared_u4(at), b = ld_shared_u4(at + 16);
        __syncwarp();
        if (lane == 0) mbar_arrive(qempty_bar(qslot));
        if (++qslot == S_QUEUE) {
            qslot = 0;
            qphase ^= 1u;
        }
        w = ScaledWork{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z};
        return w.item >= 0;
    };

    if (warp < S_EPI_WARP0) {
        if constexpr (PAIR) registers_fewer<S_OTHER_REGS>();
        if (warp == 0) {
            // -------------------------------------------------------- producer
            int stage = 0;
            uint32_t phase = 0;
            uint32_t filled = 0, fill_parity = 0;
            bool ok = true;
            const uint32_t full0_c = PAIR ? mapa_shared(full_bar(0), 0) : 0u;
            while (ok && next_work()) {
                const int l0 = (w.tm * Cf::CM + rank) * 128;
                const int cols = p.s.width / Cf::CM;  // this CTA's columns
                const int r0 = w.n0 + rank * cols;
                const uint32_t r_bytes = p.r_mn ? (uint32_t)Cf::R_BYTES : (uint32_t)cols * S_BK;
                for (int kb = w.k0; kb < w.k1; ++kb) {
                    if (!__all_sync(0xffffffffu, wait(empty_bar(stage), phase ^ 1u))) {
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
                // 64 columns: of 128 bytes a row, or rows of 128 bytes
                const uint64_t r_part = p.r_mn ? 64 >> 4 : (64 * 128) >> 4;
                while (ok && next_work()) {
                    const uint32_t idesc = p.idesc | ((uint32_t)(p.s.width / Cf::PRODUCTS >> 3) << 17);
                    for (int kb = w.k0; kb < w.k1; ++kb) {
                        // the barriers' states are asked for together, as each answer takes
                        // some hundred cycles, and waited for where one is not ready
                        bool here = mbar_test(full_bar(stage), phase);
                        bool free[Cf::PRODUCTS];
#pragma unroll
                        for (int h = 0; h < Cf::PRODUCTS; ++h) free[h] = mbar_test(tempty_bar(h * BUFFERS + buf), tphase ^ 1u);
                        if (!here) here = wait(full_bar(stage), phase);
                        const uint64_t at = (uint64_t)((uint32_t)(stage * Cf::STAGE_BYTES) >> 4);
                        auto issue = [&](int h) {  // one lane
                            const int b = h * BUFFERS + buf;
                            const uint32_t d_tmem = tmem_base + (uint32_t)(b * 128);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                const uint64_t ld = l_desc0 + at + (uint64_t)kk * l_step;
                                const uint64_t rd = r_desc0 + at + (uint64_t)h * r_part + (uint64_t)kk * r_step;
                                if constexpr (PAIR) mma_f8_ss_pair(d_tmem, ld, rd, idesc, kk > 0);
                                else mma_f8_ss(d_tmem, ld, rd, idesc, kk > 0);
                            }
                            if constexpr (PAIR) {
                                mma_commit_pair_multicast(tfull_bar(b), PAIR_MASK);
                                if (h == Cf::PRODUCTS - 1) mma_commit_pair_multicast(empty_bar(stage), PAIR_MASK);
                            } else {
                                mma_commit(tfull_bar(b));
                                mma_commit(empty_bar(stage));
                            }
                        };
                        if (!free[0]) here = here && wait(tempty_bar(buf), tphase ^ 1u);
                        const bool both = PAIR && free[Cf::PRODUCTS - 1];
                        ok = __all_sync(0xffffffffu, here);
                        if (!ok) break;
                        const bool at_once = __all_sync(0xffffffffu, both);
                        tc_fence_after_sync();
                        if (elect_one()) {
                            issue(0);
                            if (PAIR && at_once) issue(Cf::PRODUCTS - 1);
                        }
                        __syncwarp();
                        if (PAIR && !at_once) {
                            ok = __all_sync(0xffffffffu, wait(tempty_bar((Cf::PRODUCTS - 1) * BUFFERS + buf), tphase ^ 1u));
                            if (!ok) break;
                            tc_fence_after_sync();
                            if (elect_one()) issue(Cf::PRODUCTS - 1);
                            __syncwarp();
                        }
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        if (++buf == BUFFERS) {
                            buf = 0;
                            tphase ^= 1u;
                        }
                    }
                    if (!ok && lane == 0) fail_pipe();
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
        } else if (warp == 2) {
            // -------------------------------------------------------- scales
            // four bytes a copy: rows of scales start anywhere
            int slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            constexpr int PER = COL_VECTOR ? Cf::TILE_N / 32 : 1;
            while (ok && next_work()) {
                const float* ls[4];
                const float* rs[PER];
                // rows and columns past the end read the last one's
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int l = min((w.tm * Cf::CM + rank) * 128 + i * 32 + lane, p.l.rows - 1);
                    ls[i] = p.l.s + (int64_t)(l >> p.l.shift) * p.l.row + (int64_t)w.k0 * p.l.group;
                }
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int c = min(w.n0 + (COL_VECTOR ? i * 32 + lane : (lane & (Cf::CM - 1)) * 128), p.r.rows - 1);
                    rs[i] = p.r.s + (int64_t)(c >> p.r.shift) * p.r.row + (int64_t)w.k0 * p.r.group;
                }
                for (int kb0 = w.k0; kb0 < w.k1; kb0 += Cf::GROUPS) {
                    if (!__all_sync(0xffffffffu, wait(sempty_bar(slot), phase ^ 1u))) {
                        if (lane == 0) fail_pipe();
                        ok = false;
                        break;
                    }
                    uint32_t at = slots + (uint32_t)(slot * Cf::SLOT_BYTES) + (uint32_t)lane * 4;
#pragma unroll 1
                    for (int kb = kb0; kb < min(kb0 + Cf::GROUPS, w.k1); ++kb) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            cp_async_4(at + i * 128, ls[i]);
                            ls[i] += p.l.group;
                        }
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            if (COL_VECTOR ? i * 32 < p.s.width : lane < Cf::CM) cp_async_4(at + S_COL_SCALES + i * 128, rs[i]);
                            rs[i] += p.r.group;
                        }
                        at += Cf::SCALE_BYTES;
                    }
                    cp_async_arrive(sfull_bar(slot));
                    if (++slot == S_SLOTS) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            cp_async_wait_all();  // the copies are complete before the CTA ends
        } else if (warp == 3) {
            // -------------------------------------------------------- scheduler
            bool more = true;
            for (int32_t step = 0; more; ++step) {
                more = scaled_work(p.s, unit, step, w);
                if (!more) w.item = -1;
                if (!__all_sync(0xffffffffu, wait(qempty_bar(qslot), qphase ^ 1u))) {
                    if (lane == 0) fail_pipe();
                    break;
                }
                if (lane == 0) {
                    const uint32_t at = queue + (uint32_t)qslot * 32u;
                    st_shared_u4(at, w.item, w.shares, w.tm, w.n0);
                    st_shared_u4(at + 16, w.valid, w.k0, w.k1, 0);
                    mbar_arrive(qfull_bar(qslot));
                    if (more && w.shares > 1 && w.item == unit)  // this unit has the first share
                        grouped_open_counter(p.counters + (size_t)unit * Cf::CM + rank, grouped_tag(p.epoch, p.status));
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
        if constexpr (PAIR) registers_more<S_EPI_REGS>();
        const int q = warp & 3;  // tensor-memory lanes 32q .. 32q + 31
        const int part = (warp - S_EPI_WARP0) >> 2;
        const int et = threadIdx.x - S_EPI_WARP0 * 32;
        const uint64_t tag = grouped_tag(p.epoch, p.status);
        const bool give_up = p.status[G_WORD_GIVE_UP] == unit + 1;
        const int first_buf = PAIR ? part * BUFFERS : 0;
        const uint32_t full0 = tfull_bar(first_buf);
        const uint32_t release0 = PAIR ? mapa_shared(tempty_bar(first_buf), 0) : tempty_bar(0);
        int buf = 0, slot = 0;
        uint32_t tphase = 0, sphase = 0;
        while (next_work()) {
            // this warp's columns: c0 .. c0 + S_CHUNK * chunks - 1 of the tile, from t0 on of
            // a product's in tensor memory
            const int wide = PAIR ? PART : (p.s.width / 2 + 15) & ~15;
            const int c0 = PAIR ? part * 64 : part * wide;
            const int t0 = PAIR ? 0 : c0;
            const int chunks = !TURNED ? PART / S_CHUNK : max(0, min(p.s.width - c0, wide)) >> 4;
            const int l = (w.tm * Cf::CM + rank) * 128 + q * 32 + lane;
            float acc[PART];
#pragma unroll
            for (int i = 0; i < PART; ++i) acc[i] = 0.f;
            bool ok = !give_up;
            const uint32_t tmem_lanes = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(first_buf * 128 + t0);
            // the answer whether a product is there is asked for before the sums of the one
            // before, as it takes some hundred cycles
            bool here = mbar_test(full0 + 8u * (uint32_t)buf, tphase);
            auto block = [&](uint32_t my_scales) {
                if (!here) ok = ok && wait(full0 + 8u * (uint32_t)buf, tphase);
                __syncwarp();
                tc_fence_after_sync();
                const uint32_t tbase = tmem_lanes + (uint32_t)(buf * 128);
                // the lane's scale, or its products with those of the columns
                const uint32_t my_cols = my_scales + S_COL_SCALES + (uint32_t)c0 * 4;
                float factors[Cf::CM];
                auto release = [&]() {  // the product has been read, by all lanes (wait::ld is the warp's)
                    tc_fence_before_sync();
                    if constexpr (PAIR) mbar_arrive_cluster_if(lane == 0, release0 + 8u * (uint32_t)buf);
                    else mbar_arrive_if(lane == 0, release0 + 8u * (uint32_t)buf);
                    if (++buf == BUFFERS) {
                        buf = 0;
                        tphase ^= 1u;
                    }
                    here = mbar_test(full0 + 8u * (uint32_t)buf, tphase);
                };
                // Columns read from tensor memory at once: a load takes some 100 cycles, whatever
                // its size, so many; but few where each column's scale is read from shared
                // memory beside them, and then one batch is read while the one before is added.
                // us, 16 against 64 at once: 8192 x 14336 x 4096 with blocks 368 / 356, with
                // vectors 496 / 561.
                constexpr int BATCH = COL_VECTOR ? 16 : 64, BATCHES = PART / BATCH, READS = COL_VECTOR ? 2 : 1;
                const int batches = TURNED ? chunks : BATCHES;
                uint32_t v[READS][BATCH];
                if (batches > 0) tmem_ld_async(tbase, v[0]);
                const float mine = ld_shared_f1(my_scales + (uint32_t)(q * 32 + lane) * 4);
#pragma unroll
                for (int i = 0; i < Cf::CM; ++i) {
                    factors[i] = mine;
                    if constexpr (!COL_VECTOR) factors[i] *= ld_shared_f1(my_scales + S_COL_SCALES + (uint32_t)((c0 >> 7) + i) * 4);
                }
#pragma unroll
                for (int b = 0; b < BATCHES; ++b) {
                    if (b < batches) {
                        uint32_t (&r)[BATCH] = v[b % READS];
                        if (READS == 1 && b > 0) tmem_ld_async(tbase + b * BATCH, r);
                        // (the scales' latency passes while the columns are on their way)
                        float4 f[COL_VECTOR ? BATCH / 4 : 1];
                        if constexpr (COL_VECTOR)
#pragma unroll
                            for (int i = 0; i < BATCH; i += 4) {
                                const int at = b * BATCH + i;
                                f[i / 4] = ld_shared_f4(my_cols + (uint32_t)(at + (PAIR && at >= 64 ? 64 : 0)) * 4);
                            }
                        tmem_wait(r);
                        if (READS == 2 && b + 1 < BATCHES && b + 1 < batches) tmem_ld_async(tbase + (b + 1) * BATCH, v[(b + 1) % READS]);
                        if (!TURNED && b == BATCHES - 1) release();
#pragma unroll
                        for (int i = 0; i < BATCH; i += 4) {
                            const int at = b * BATCH + i;
                            const float factor = factors[PAIR && at >= 64 ? 1 : 0];
                            scaled_add4<COL_VECTOR>(acc + at, r + i, COL_VECTOR ? f[i / 4] : make_float4(factor, factor, factor, factor), factor);
                        }
                    }
                }
                if (TURNED) release();
            };
#pragma unroll 1
            for (int kb0 = w.k0; kb0 < w.k1; kb0 += Cf::GROUPS) {
                ok = ok && wait(sfull_bar(slot), sphase);
                uint32_t my_scales = slots + (uint32_t)(slot * Cf::SLOT_BYTES);
                const int n = min(Cf::GROUPS, w.k1 - kb0);
#pragma unroll 1
                for (int i = 0; i < n; ++i, my_scales += Cf::SCALE_BYTES) block(my_scales);
                __syncwarp();
                mbar_arrive_if(lane == 0, sempty_bar(slot));
                if (++slot == S_SLOTS) {
                    slot = 0;
                    sphase ^= 1u;
                }
            }
            if (!ok && lane == 0) fail_pipe();
            // (a warp that gives up must not leave the others at a barrier)
            if (!scaled_vote_all(ok)) break;
            if (w.shares > 1) {
                float4* mine = reinterpret_cast<float4*>(p.partials + (size_t)blockIdx.x * Cf::SLOT_FLOATS) + et;
#pragma unroll
                for (int i = 0; i < PART / 4; ++i)
                    if (i < chunks * (S_CHUNK / 4))
                        st_f4(mine + i * S_EPI_THREADS, make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]));
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
                for (int i = 0; i < PART; ++i) acc[i] = 0.f;
#pragma unroll 1
                for (int x = 0; x < w.shares; ++x) {
                    // share x was run by unit w.item + x
                    const float4* from = reinterpret_cast<const float4*>(
                        p.partials + (size_t)((w.item + x) * Cf::CM + rank) * Cf::SLOT_FLOATS) + et;
#pragma unroll
                    for (int i = 0; i < PART / 4; ++i)
                        if (i < chunks * (S_CHUNK / 4)) {
                            const float4 y = ld_cg_f4(from + i * S_EPI_THREADS);
                            acc[4 * i] += y.x;
                            acc[4 * i + 1] += y.y;
                            acc[4 * i + 2] += y.z;
                            acc[4 * i + 3] += y.w;
                        }
                }
            }
            // ---- the tile to C
            if (!TURNED && p.boxes) {
                // by tensor copies of boxes of 32 rows x 64 bytes, 16-byte units swizzled by
                // row.  (Stored by the lanes, a row each, an instruction touches 32 lines:
                // some 4000 cycles a tile.)
                constexpr int B = Cf::BOXES;
                const uint32_t my_box = boxes + (uint32_t)((warp - S_EPI_WARP0) * B) * 2048u;
                int box = 0;
                auto stage = [&](int x, const uint32_t (&u)[16]) {  // 64 bytes of the lane's row
                    if (lane == 0) bulk_wait_group_read<(B > 0 ? B - 1 : 0)>();
                    __syncwarp();
                    const uint32_t at = my_box + (uint32_t)box * 2048u;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        st_shared_u4(at + (uint32_t)lane * 64u + (uint32_t)((i ^ ((lane >> 1) & 3)) * 16), u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (x < (int)p.ldc && l < p.l_total) tma_store_2d(&tm.c, at, x, l);
                        bulk_commit_group();
                    }
                    box = box + 1 == B ? 0 : box + 1;
                };
                if (p.out_dtype == 2) {
#pragma unroll
                    for (int i = 0; i < PART; i += 16) {
                        uint32_t u[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(acc[i + j]);
                        stage(w.n0 + c0 + i + (PAIR && i >= 64 ? 64 : 0), u);
                    }
                } else {
                    const bool bf16 = p.out_dtype == 1;
#pragma unroll
                    for (int i = 0; i < PART; i += 32) {
                        uint32_t u[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j] = scaled_pack2(bf16, acc[i + 2 * j], acc[i + 2 * j + 1]);
                        stage(w.n0 + c0 + i + (PAIR && i >= 64 ? 64 : 0), u);
                    }
                }
                continue;
            }
            if (l >= p.l_total) continue;
            if constexpr (TURNED) {
                // a column is a row of C: 32 lanes store neighbours
                const int count = min(w.valid - c0, chunks * S_CHUNK);
                const int64_t at = (int64_t)(w.n0 + c0) * p.ldc + l;
                if (p.out_dtype == 2) {
                    float* out = static_cast<float*>(p.out) + at;
#pragma unroll
                    for (int i = 0; i < PART; ++i)
                        if (i < count) out[(int64_t)i * p.ldc] = acc[i];
                } else {
                    const bool bf16 = p.out_dtype == 1;
                    uint16_t* out = static_cast<uint16_t*>(p.out) + at;
#pragma unroll
                    for (int i = 0; i < PART; ++i)
                        if (i < count) out[(int64_t)i * p.ldc] = (uint16_t)scaled_pack2(bf16, acc[i], 0.f);
                }
            } else {
                // rows of C that tensor copies cannot address: element by element
                const int64_t at = (int64_t)l * p.ldc + w.n0 + c0;
#pragma unroll
                for (int i = 0; i < PART; ++i) {
                    const int c = i + (PAIR && i >= 64 ? 64 : 0);
                    if (c0 + c < w.valid) scaled_store(p.out, p.out_dtype, at + c, acc[i]);
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
