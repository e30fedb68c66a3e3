// Tile scheduler of the grouped products: which output tiles and k-ranges a
// scheduling unit (a CTA, or a pair of CTAs) runs.  Host and device run the
// same code; the group sizes are known on the device only, so every CTA
// derives the tile table from the offsets at its start.
//
// A tile has tile_m columns of a matrix along the tensor memory's lanes and up
// to tile_n rows along its columns.  ROWS: the rows of a group are cut into
// ceil(n / tile_n) tiles of one width, the smallest multiple of `step` that
// covers them, so a group wastes at most step - 1 rows of tensor work a tile.
// INNER: the output matrices are cut into full tiles and the group's rows are
// the summed dimension.
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
    int32_t tile_n, step;
    int32_t band;          // raster: tiles along the columns side visited before the next lanes tile
    int32_t units;         // scheduling units
    int32_t min_iters;     // least k-blocks of a split share
};

// off[0 .. groups]: bounded offsets; first[0 .. groups]: tiles before a group.
struct GroupedTables {
    const int32_t* off;
    const int32_t* first;
};

__host__ __device__ __forceinline__ int32_t grouped_tiles_of(const GroupedShape& s, int32_t n) {
    return s.inner ? s.tiles_m * s.tiles_n : s.tiles_m * ((n + s.tile_n - 1) / s.tile_n);
}

// A unit of work: k-blocks [k0, k1) of the kb of one tile.
struct GroupedWork {
    int32_t tile, group, tm;
    int32_t n0;       // first row of the tile: of A (ROWS), of the output matrix (INNER)
    int32_t width;    // columns of the accumulator
    int32_t valid;    // rows to store
    int32_t r0, r1;   // the group's rows
    int32_t k0, k1, kb;
};

struct GroupedCursor {
    int32_t tiles, split_tiles;  // all tiles; the first split_tiles of them are split by k
    int32_t split_units;
    int64_t q, r;                // split k-blocks a unit: q, one more for the first r
    int64_t it, it_end;          // this unit's split k-blocks
    int32_t next_tile, group;
};

__host__ __device__ __forceinline__ void grouped_cursor_init(const GroupedShape& s, const GroupedTables& t,
                                                             int32_t unit, GroupedCursor& c) {
    c.tiles = t.first[s.groups];
    c.group = 0;
    // Under one wave of tiles, all are split evenly over the units by k;
    // otherwise all tiles run whole.
    c.split_tiles = (!s.inner && c.tiles < s.units) ? c.tiles : 0;
    const int64_t total = (int64_t)c.split_tiles * s.kb;
    const int64_t want = total / s.min_iters;
    c.split_units = want < 1 ? 1 : (want < s.units ? (int32_t)want : s.units);
    c.q = total / c.split_units;
    c.r = total % c.split_units;
    if (unit < c.split_units) {
        c.it = unit * c.q + (unit < c.r ? unit : c.r);
        c.it_end = c.it + c.q + (unit < c.r ? 1 : 0);
    } else {
        c.it = c.it_end = 0;
    }
    c.next_tile = c.split_tiles + unit;
}

// The unit that runs split k-block `it`.
__host__ __device__ __forceinline__ int32_t grouped_split_unit(const GroupedCursor& c, int64_t it) {
    const int64_t big = c.r * (c.q + 1);
    return (int32_t)(it < big ? it / (c.q + 1) : c.r + (it - big) / c.q);
}

__host__ __device__ __forceinline__ bool grouped_cursor_next(const GroupedShape& s, const GroupedTables& t,
                                                             GroupedCursor& c, GroupedWork& w) {
    int32_t tile, k0 = 0, k1 = -1;
    if (c.it < c.it_end) {
        tile = (int32_t)(c.it / s.kb);
        k0 = (int32_t)(c.it % s.kb);
        k1 = (int32_t)(k0 + (c.it_end - c.it));
        if (k1 > s.kb) k1 = s.kb;
        c.it += k1 - k0;
    } else if (c.next_tile < c.tiles) {
        tile = c.next_tile;
        c.next_tile += s.units;
    } else {
        return false;
    }
    while (tile >= t.first[c.group + 1]) ++c.group;
    const int32_t g = c.group;
    w.tile = tile;
    w.group = g;
    w.r0 = t.off[g];
    w.r1 = t.off[g + 1];
    const int32_t n = w.r1 - w.r0;
    const int32_t side = s.inner ? s.tiles_n : (n + s.tile_n - 1) / s.tile_n;
    // bands of `band` tiles along the columns side, the lanes side slow within one
    const int32_t local = tile - t.first[g];
    const int32_t b = local / (s.band * s.tiles_m), in = local - b * s.band * s.tiles_m;
    const int32_t wide = side - b * s.band < s.band ? side - b * s.band : s.band;
    w.tm = in / wide;
    const int32_t tn = b * s.band + in % wide;
    if (s.inner) {
        w.width = s.tile_n;
        w.n0 = tn * s.tile_n;
        w.valid = s.n_total - w.n0 < s.tile_n ? s.n_total - w.n0 : s.tile_n;
        w.kb = (n + 63) / 64;
    } else {
        w.width = ((n + side - 1) / side + s.step - 1) / s.step * s.step;
        w.n0 = w.r0 + tn * w.width;
        w.valid = w.r1 - w.n0 < w.width ? w.r1 - w.n0 : w.width;
        w.kb = s.kb;
    }
    w.k0 = k0;
    w.k1 = k1 < 0 ? w.kb : k1;
    return true;
}

}  // namespace psm
