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
// Split.  Tiles that do not fill a round of the units (all of them when there
// are fewer than units, else, for ROWS, the remainder) run first, the k-blocks
// of each cut into near-equal shares, each share run by a unit of its own:
// ceil(kb / L) of them, with L k-blocks a share at most, chosen so that the
// shares fit the units.  A unit never has more than one share, so it never
// joins one tile while another waits; what it has after it are whole tiles,
// which hide the joining.  us with the remainder whole against split: 79 / 55
// (2 groups, 4096 rows of 8192, 85 tiles for 76 pairs), 59 / 46 (13 groups,
// 1482 rows of 5952 x 1424), 43.6 / 34.5 (one group, 1024 rows of 4096 x 5120),
// 68.5 / 65.9 (64 groups of 2048 x 1536), the same where the shares would be
// too short.
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
// g = 0 .. groups, of their items: tiles, or for a split INNER shares of tiles.
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

struct GroupedSplit {
    int32_t tiles;   // the first tiles are split
    int32_t most;    // k-blocks of a share at most; 0: no split
    int32_t shares;  // ROWS: shares of each
};

// For all tiles and (INNER) their k-blocks.  The sum over the split tiles of
// ceil(kb / L) is at most total / L + tiles, so this L keeps it within the units.
__host__ __device__ __forceinline__ GroupedSplit grouped_split(const GroupedShape& s, int32_t tiles, int32_t blocks) {
    GroupedSplit p{0, 0, 1};
    const int32_t rest = tiles < s.units ? tiles : (s.inner ? 0 : tiles % s.units);
    if (!s.may_split || rest == 0 || (!s.inner && s.kb <= s.least_share)) return p;
    const int32_t total = s.inner ? blocks : rest * s.kb;
    const int32_t l = (int32_t)(((uint32_t)total + (uint32_t)(s.units - rest) - 1u) / (uint32_t)(s.units - rest));
    const int32_t most = l > s.least_share ? l : s.least_share;
    const int32_t shares = s.inner ? 1 : grouped_shares(s.kb, most);
    if (s.inner || shares > 1) p = GroupedSplit{rest, most, shares};
    return p;
}

// A unit of work: k-blocks [k0, k1) of the kb of one tile.
struct GroupedWork {
    int32_t item;     // split: the unit of the first share, the others' follow; else the tile
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

// The unit's work number `step`; false past its last.  `items`: first[groups].
__host__ __device__ __forceinline__ bool grouped_work(const GroupedShape& s, const GroupedTables& t,
                                                      const GroupedSplit& p, int32_t unit, int32_t step,
                                                      int32_t items, GroupedWork& w) {
    uint32_t next;       // the tile, or for INNER the share; below 2^32, as the one before is below 2^31
    int32_t share = 0;
    w.shares = 1;
    if (!s.inner && p.most > 0) {
        const bool has = unit < p.tiles * p.shares;
        if (has && step == 0) {
            next = (uint32_t)(unit / p.shares);
            share = unit - (int32_t)next * p.shares;
            w.shares = p.shares;
        } else {
            next = (uint32_t)p.tiles + (uint32_t)unit + (uint32_t)(step - has) * (uint32_t)s.units;
        }
    } else {
        next = (uint32_t)unit + (uint32_t)step * (uint32_t)s.units;
    }
    if (next >= (uint32_t)items) return false;
    const int32_t at = (int32_t)next;
    const int32_t g = grouped_search(s.groups, at, t.first);
    w.group = g;
    w.r0 = t.off[g];
    w.r1 = t.off[g + 1];
    const int32_t n = w.r1 - w.r0;
    w.kb = grouped_k_blocks(s, n);
    int32_t local = at - t.first[g];
    w.item = at;
    if (s.inner && p.most > 0) {
        w.shares = grouped_shares(w.kb, p.most);
        if (w.shares > 1) {
            const int32_t tile = local / w.shares;
            share = local - tile * w.shares;
            local = tile;
        }
        w.item = at - share;
    } else if (w.shares > 1) {
        w.item = unit - share;
    }
    w.k0 = w.shares > 1 ? (int32_t)((int64_t)w.kb * share / w.shares) : 0;
    w.k1 = w.shares > 1 ? (int32_t)((int64_t)w.kb * (share + 1) / w.shares) : w.kb;
    const int32_t side = s.inner ? s.tiles_n : (n + s.tile_n - 1) >> s.tile_shift;
    // bands of about `band` tiles along the columns side, even ones (with eight
    // and a rest of one, nine tiles of rows read the matrix twice), the lanes
    // side slow within one
    int32_t first_tn = 0, wide = side;
    if (2 * side > 3 * s.band) {
        const int32_t bands = (side + s.band / 2 - 1) / s.band;
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
        // the even part, rounded up (n > 0; n + side - 1 may pass 2^31)
        w.width = ((side == 1 ? n : (n - 1) / side + 1) + s.step - 1) & ~(s.step - 1);
        w.n0 = w.r0 + tn * w.width;
        w.valid = w.r1 - w.n0 < w.width ? w.r1 - w.n0 : w.width;
    }
    return true;
}

}  // namespace psm
