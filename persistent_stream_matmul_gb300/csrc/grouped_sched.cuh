// Tile scheduler of the grouped products: which output tiles and k-ranges a
// scheduling unit (a CTA, or a pair of CTAs) runs.  Host and device run the
// same code; the group sizes are known on the device only, so every CTA
// derives the tile tables from the offsets at its start.
//
// A tile has tile_m columns of a matrix along the tensor memory's lanes and up
// to tile_n rows along its columns.  ROWS: the rows of a group are cut into
// ceil(n / tile_n) tiles of one width, the smallest multiple of `step` that
// covers them, so a group wastes at most step - 1 rows of tensor work a tile.
// INNER: the output matrices are cut into full tiles and the group's rows are
// the summed dimension.
//
// Order.  Tiles run in the order of their groups.  (Spreading the tiles of
// groups with few rows, which are bound by memory, evenly among the others
// changed 24006 skewed rows over 64 groups by less than 1 %.)
//
// Split.  With fewer tiles than units, the k-blocks of all tiles are split
// evenly over units; a share may end inside a tile and the next begin there.
#pragma once
#include <stdint.h>

namespace psm {

struct GroupedShape {
    int32_t groups, rows;
    int32_t inner;         // 0: ROWS, 1: INNER
    int32_t tiles_m;       // tiles along the lanes side
    int32_t tiles_n;       // INNER: tiles along the other side of the output
    int32_t n_total;       // INNER: extent of that side
    int32_t kb;            // ROWS: k-blocks of 64 a tile
    int32_t tile_n, step;  // tile_n: 1 << tile_shift; step a power of two
    int32_t tile_shift;
    int32_t band;          // raster: tiles along the columns side visited before the next lanes tile
    int32_t units;         // scheduling units
    int32_t may_split;     // the k-blocks of fewer than `units` tiles fit an int32
};

// off[0 .. groups]: bounded offsets.  Sums over the groups before g, for g =
// 0 .. groups: tiles, and (INNER) k-blocks of the tiles.
struct GroupedTables {
    const int32_t* off;
    const int32_t* first;
    const int32_t* iters;
};

struct GroupedCounts {
    int32_t tiles, iters;
};

__host__ __device__ __forceinline__ GroupedCounts grouped_counts(const GroupedShape& s, int32_t n) {
    GroupedCounts c;
    c.tiles = s.inner ? s.tiles_m * s.tiles_n : s.tiles_m * ((n + s.tile_n - 1) >> s.tile_shift);
    c.iters = s.inner && s.may_split ? c.tiles * ((n + 63) / 64) : 0;
    return c;
}

// A unit of work: k-blocks [k0, k1) of the kb of one tile.
struct GroupedWork {
    int32_t tile;
    int32_t it0;      // its first k-block among all split ones
    int32_t group, tm;
    int32_t n0;       // first row of the tile: of A (ROWS), of the output matrix (INNER)
    int32_t width;    // columns of the accumulator
    int32_t valid;    // rows to store
    int32_t r0, r1;   // the group's rows
    int32_t k0, k1, kb;
};

struct GroupedCursor {
    int32_t tiles;
    bool split;
    int32_t q, r;                // split k-blocks a unit: q, one more for the first r
    int32_t it, it_end;          // this unit's split k-blocks
    int32_t next_tile;
};

__host__ __device__ __forceinline__ void grouped_cursor_init(const GroupedShape& s, const GroupedTables& t,
                                                             int32_t unit, GroupedCursor& c) {
    c.tiles = t.first[s.groups];
    c.split = s.may_split && c.tiles < s.units;
    c.q = c.r = c.it = c.it_end = 0;
    c.next_tile = c.split && !s.inner ? c.tiles : unit;
    if (c.split && c.tiles > 0) {
        // A share costs its k-blocks, and the contributor that joins a tile
        // reads every share's partial, worth about 4 k-blocks of the widest
        // tile: the joined time is least near sqrt(k-blocks) / 2 shares a
        // tile.  Narrow tiles, bound by the reads of the matrix, bear twice that.
        const int32_t total = s.inner ? t.iters[s.groups] : c.tiles * s.kb;
        const int32_t mean = s.inner ? total / c.tiles : s.kb;
        int32_t shares = 1;
        while (shares < 32 && (shares + 1) * (shares + 1) <= (s.step == 16 ? mean : mean / 4)) ++shares;
        const int32_t n = c.tiles * shares < s.units ? c.tiles * shares : s.units;
        c.q = total / n;
        c.r = total - c.q * n;
        if (unit < n) {
            c.it = unit * c.q + (unit < c.r ? unit : c.r);
            c.it_end = c.it + c.q + (unit < c.r ? 1 : 0);
        }
    }
}

// The unit that runs split k-block `it`, for a cursor's q and r.
__host__ __device__ __forceinline__ int32_t grouped_split_unit(int32_t q, int32_t r, int32_t it) {
    const int32_t big = r * (q + 1);
    return it < big ? it / (q + 1) : r + (it - big) / q;
}

// The group g with sum[g] <= x < sum[g + 1].
__host__ __device__ __forceinline__ int32_t grouped_search(int32_t groups, int32_t x, const int32_t* sum) {
#ifdef __CUDA_ARCH__
    const int lane = threadIdx.x & 31;
    int32_t base = 0;
    if (groups > 32) {
        const int32_t i = lane * 32;
        base = 32 * (__popc(__ballot_sync(0xffffffffu, i < groups && sum[i] <= x)) - 1);
    }
    const int32_t i = base + lane;
    return base + __popc(__ballot_sync(0xffffffffu, i < groups && sum[i] <= x)) - 1;
#else
    int32_t lo = 0, hi = groups;  // sum[lo] <= x < sum[hi]
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (sum[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
#endif
}

__host__ __device__ __forceinline__ bool grouped_cursor_next(const GroupedShape& s, const GroupedTables& t,
                                                             GroupedCursor& c, GroupedWork& w) {
    int32_t g, local;  // group, and tile within it
    while (true) {
        w.k0 = 0;
        w.k1 = -1;
        if (c.it < c.it_end) {
            w.k1 = c.it_end - c.it;  // an upper bound, from k0
            if (s.inner) {
                g = grouped_search(s.groups, c.it, t.iters);
                const int32_t kb = (t.off[g + 1] - t.off[g] + 63) / 64;
                local = (c.it - t.iters[g]) / kb;
                w.it0 = t.iters[g] + local * kb;
                w.tile = t.first[g] + local;
            } else {
                w.tile = c.it / s.kb;
                w.it0 = w.tile * s.kb;
                g = grouped_search(s.groups, w.tile, t.first);
                local = w.tile - t.first[g];
            }
            w.k0 = c.it - w.it0;
        } else if (c.next_tile < c.tiles) {
            w.tile = c.next_tile;
            c.next_tile += s.units;
            w.it0 = 0;
            g = grouped_search(s.groups, w.tile, t.first);
            local = w.tile - t.first[g];
            // INNER: a split leaves the tiles of empty groups to be cleared
            if (c.split && t.off[g + 1] > t.off[g]) continue;
        } else {
            return false;
        }
        break;
    }
    w.group = g;
    w.r0 = t.off[g];
    w.r1 = t.off[g + 1];
    const int32_t n = w.r1 - w.r0;
    const int32_t side = s.inner ? s.tiles_n : (n + s.tile_n - 1) >> s.tile_shift;
    // bands of `band` tiles along the columns side, the lanes side slow within
    // one; without the divisions that the common shapes do not need
    int32_t first_tn = 0, wide = side;
    if (side > s.band) {
        const int32_t b = local / (s.band * s.tiles_m);
        local -= b * s.band * s.tiles_m;
        first_tn = b * s.band;
        wide = side - first_tn < s.band ? side - first_tn : s.band;
    }
    w.tm = wide == 1 ? local : local / wide;
    const int32_t tn = first_tn + local - w.tm * wide;
    if (s.inner) {
        w.width = s.tile_n;
        w.n0 = tn * s.tile_n;
        w.valid = s.n_total - w.n0 < s.tile_n ? s.n_total - w.n0 : s.tile_n;
        w.kb = (n + 63) / 64;
    } else {
        w.width = ((side == 1 ? n : (n + side - 1) / side) + s.step - 1) & ~(s.step - 1);
        w.n0 = w.r0 + tn * w.width;
        w.valid = w.r1 - w.n0 < w.width ? w.r1 - w.n0 : w.width;
        w.kb = s.kb;
    }
    if (w.k1 < 0 || w.k0 + w.k1 > w.kb) w.k1 = w.kb;
    else w.k1 += w.k0;
    if (c.it < c.it_end) c.it += w.k1 - w.k0;
    return true;
}

}  // namespace psm
