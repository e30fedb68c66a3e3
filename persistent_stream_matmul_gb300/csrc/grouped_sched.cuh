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
// Split.  With fewer tiles than units, the k-blocks of a tile are cut into
// near-equal shares, each run by a unit of its own: ceil(kb / L) of them, with
// L k-blocks a share at most, chosen so that the shares of all tiles fit the
// units.  A unit never has more than one share, so it never joins one tile
// while another waits.
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
    int32_t band;          // raster: about how many tiles along the columns side are visited before
                           // the next lanes tile
    int32_t units;         // scheduling units
    int32_t may_split;     // the k-blocks of fewer than `units` tiles fit an int32
    int32_t least_share;   // least k-blocks of a share worth joining
};

// off[0 .. groups]: bounded offsets.  first: sums over the groups before g, for
// g = 0 .. groups, of their items: tiles, or shares of tiles once split.
struct GroupedTables {
    const int32_t* off;
    int32_t* first;
};

__host__ __device__ __forceinline__ int32_t grouped_tiles(const GroupedShape& s, int32_t n) {
    return s.inner ? s.tiles_m * s.tiles_n : s.tiles_m * ((n + s.tile_n - 1) >> s.tile_shift);
}

__host__ __device__ __forceinline__ int32_t grouped_k_blocks(const GroupedShape& s, int32_t n) {
    return s.inner ? (n + 63) / 64 : s.kb;
}

// Shares of a tile of kb k-blocks, at most `most` each (0: not split).
__host__ __device__ __forceinline__ int32_t grouped_shares(int32_t kb, int32_t most) {
    return most == 0 || kb <= most ? 1 : (kb + most - 1) / most;
}

// The k-blocks of a share at most, for all tiles and the k-blocks of all tiles
// (0: no split).  sum over tiles of ceil(kb / L) <= total / L + tiles, so this L
// keeps the shares within the units.
__host__ __device__ __forceinline__ int32_t grouped_share_limit(const GroupedShape& s, int32_t tiles, int32_t total) {
    if (!s.may_split || tiles == 0 || tiles >= s.units) return 0;
    const int32_t l = (total + s.units - tiles - 1) / (s.units - tiles);
    return l > s.least_share ? l : s.least_share;
}

// A unit of work: k-blocks [k0, k1) of the kb of one tile.
struct GroupedWork {
    int32_t item;     // of the tile's first share; the others follow
    int32_t shares;
    int32_t group, tm;
    int32_t n0;       // first row of the tile: of A (ROWS), of the output matrix (INNER)
    int32_t width;    // columns of the accumulator
    int32_t valid;    // rows to store
    int32_t r0, r1;   // the group's rows
    int32_t k0, k1, kb;
};

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

// Work item `item`, for shares of at most `most` k-blocks.
__host__ __device__ __forceinline__ void grouped_work(const GroupedShape& s, const GroupedTables& t, int32_t most,
                                                      int32_t item, GroupedWork& w) {
    const int32_t g = grouped_search(s.groups, item, t.first);
    w.group = g;
    w.r0 = t.off[g];
    w.r1 = t.off[g + 1];
    const int32_t n = w.r1 - w.r0;
    w.kb = grouped_k_blocks(s, n);
    w.shares = grouped_shares(w.kb, most);
    int32_t local = item - t.first[g], share = 0;
    if (w.shares > 1) {
        const int32_t tile = local / w.shares;
        share = local - tile * w.shares;
        local = tile;
    }
    w.item = item - share;
    w.k0 = w.shares > 1 ? (int32_t)((int64_t)w.kb * share / w.shares) : 0;
    w.k1 = w.shares > 1 ? (int32_t)((int64_t)w.kb * (share + 1) / w.shares) : w.kb;
    const int32_t side = s.inner ? s.tiles_n : (n + s.tile_n - 1) >> s.tile_shift;
    // bands of about `band` tiles along the columns side, even ones (with eight
    // and a rest of one, nine tiles of rows read the matrix twice), the lanes
    // side slow within one
    int32_t first_tn = 0, wide = side;
    const int32_t bands = (side + s.band / 2 - 1) / s.band;
    if (bands > 1) {
        const int32_t most_wide = (side + bands - 1) / bands;
        const int32_t b = local / (most_wide * s.tiles_m);
        local -= b * most_wide * s.tiles_m;
        first_tn = b * most_wide;
        wide = side - first_tn < most_wide ? side - first_tn : most_wide;
    }
    w.tm = wide == 1 ? local : local / wide;
    const int32_t tn = first_tn + local - w.tm * wide;
    if (s.inner) {
        w.width = s.tile_n;
        w.n0 = tn * s.tile_n;
        w.valid = s.n_total - w.n0 < s.tile_n ? s.n_total - w.n0 : s.tile_n;
    } else {
        w.width = ((side == 1 ? n : (n + side - 1) / side) + s.step - 1) & ~(s.step - 1);
        w.n0 = w.r0 + tn * w.width;
        w.valid = w.r1 - w.n0 < w.width ? w.r1 - w.n0 : w.width;
    }
}

}  // namespace psm
