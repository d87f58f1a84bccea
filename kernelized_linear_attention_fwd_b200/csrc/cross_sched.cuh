// How the tensor-core cross attention shares its work out (cross_tc.cu), and which
// pieces of an item the join adds up (cross.cu).
//
// The work of one mode is a line of units (128-row tile, 128-column block): sequence b
// has Hkv T_b N_b of them, T_b row tiles and N_b column blocks; in the forward and
// dq passes N_b follows the sequence's visible keys, in dkv T_b does.  An item is
// one tile of one head; CTA c of G takes the units [c S, (c + 1) S),
// S = max(ceil(total / G), min_share).  So every CTA has the same work whatever the
// lengths are, and few long items are split over all CTAs.  Plans whose items fill the grid many times over do not
// cut (whole): there the cuts are moved down to item boundaries.
#pragma once

#include "kata_internal.cuh"

namespace kata {

constexpr int kXCols = 128;  // columns of a block
constexpr int kXTile = 128;  // rows of a tile

// A place in the line: block `blk` of tile `p` of head `h` of sequence `b`.
struct XPos {
    int b, h, p, blk;
};
struct XRange {
    XPos from, to;
};
// What the join needs of a CTA's first piece (XIter::first): its item, whether it
// continues one that an earlier CTA began, and whether it reaches the item's end.
struct alignas(16) XPiece {
    int bh, r0;
    int cont, last;
};
// A stretch of blocks of one item.
struct XItem {
    int bh, r0, b0, n_blk;
    int cols;  // columns in use (dkv: all of them)
    int live;  // visible keys of the sequence
    int part;  // slot of a cut item's piece, or -1
    int reaches_end;
};

// T_b and N_b.
template <int MODE>
__device__ __forceinline__ void x_extent(const XSched &s, int b, int &live, int &tiles, int &blocks) {
    live = cross_length(s.key_lengths, b, s.Tk);
    const int rows = MODE == kCrossDkv ? live : s.rows, cols = MODE == kCrossDkv ? s.cols : live;
    tiles = (rows + kXTile - 1) / kXTile;
    blocks = (cols + kXCols - 1) / kXCols;
}

// Place of unit `off` of sequence b.
__device__ __forceinline__ XPos x_place(const XSched &s, int b, long long off, int tiles, int blocks) {
    const long long per_head = (long long)tiles * blocks;
    XPos r;
    r.b = b;
    r.h = (int)(off / per_head);
    const long long rem = off - r.h * per_head;
    r.p = (int)(rem / blocks);
    r.blk = s.whole ? 0 : (int)(rem - (long long)r.p * blocks);
    return r;
}

// The whole line as one warp sees it: every lane holds the units of a run of
// sequences.  Call with all 32 lanes.
template <int MODE>
struct XLine {
    long long before, units, total;  // units before this lane's run, in it, in all
    int first, last;                 // the run

    __device__ __forceinline__ XLine(const XSched &s, int lane) {
        if (!s.key_lengths) {  // all sequences alike: lane 0 holds them
            int live, tiles, blocks;
            x_extent<MODE>(s, 0, live, tiles, blocks);
            total = (long long)s.B * s.Hkv * tiles * blocks;
            units = lane == 0 ? total : 0;
            before = lane == 0 ? 0 : total;
            first = lane == 0 ? 0 : s.B;
            last = s.B;
            return;
        }
        const int run = (s.B + 31) / 32;
        first = min(s.B, lane * run);
        last = min(s.B, first + run);
        units = 0;
#pragma unroll 8
        for (int b = first; b < last; ++b) {
            int live, tiles, blocks;
            x_extent<MODE>(s, b, live, tiles, blocks);
            units += (long long)s.Hkv * tiles * blocks;
        }
        long long sum = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        before = sum - units;
        total = __shfl_sync(0xffffffffu, sum, 31);
    }

    __device__ __forceinline__ long long share(const XSched &s, int grid) const {
        const long long n = (total + grid - 1) / grid;
        return n < s.min_share ? s.min_share : n;
    }

    // Place of unit u.
    __device__ __forceinline__ XPos place(const XSched &s, long long u) const {
        XPos r = {s.B, 0, 0, 0};
        const bool mine = u < total && u >= before && u < before + units;
        if (mine) {
            long long at = before;
            if (!s.key_lengths) {
                int live, tiles, blocks;
                x_extent<MODE>(s, 0, live, tiles, blocks);
                const long long per = (long long)s.Hkv * tiles * blocks;
                const int b = (int)(u / per);
                r = x_place(s, b, u - b * per, tiles, blocks);
            } else {
                for (int b = first; b < last; ++b) {
                    int live, tiles, blocks;
                    x_extent<MODE>(s, b, live, tiles, blocks);
                    const long long per = (long long)s.Hkv * tiles * blocks;
                    if (u < at + per) {
                        r = x_place(s, b, u - at, tiles, blocks);
                        break;
                    }
                    at += per;
                }
            }
        }
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        const int src = who ? __ffs(who) - 1 : 0;
        r.b = __shfl_sync(0xffffffffu, r.b, src);
        r.h = __shfl_sync(0xffffffffu, r.h, src);
        r.p = __shfl_sync(0xffffffffu, r.p, src);
        r.blk = __shfl_sync(0xffffffffu, r.blk, src);
        return r;
    }
};

// CTA c's stretch.  All 32 lanes.
template <int MODE>
__device__ __forceinline__ XRange x_range(const XSched &s, int c, int lane) {
    const XLine<MODE> line(s, lane);
    const long long n = line.share(s, s.grid);
    XRange r;
    r.from = line.place(s, n * c);
    r.to = line.place(s, n * (c + 1));
    return r;
}

template <int MODE>
struct XIter {
    const XSched &s;
    XPos at, to;
    int cta, pieces = 0;

    __device__ __forceinline__ XIter(const XSched &s_, const XRange &r, int cta_)
        : s(s_), at(r.from), to(r.to), cta(cta_) {}

    // The first piece, of an iterator that has not started (bh = -1: none).
    __device__ __forceinline__ static XPiece first(const XSched &s, const XRange &r) {
        XIter x(s, r, 0);
        XItem it;
        if (!x.next(it)) return {-1, 0, 0, 0};
        return {it.bh, it.r0, it.b0 > 0, it.reaches_end};
    }

    __device__ __forceinline__ bool next(XItem &it) {
        while (at.b < s.B) {
            if (at.b == to.b && at.h == to.h && at.p == to.p && at.blk == to.blk) return false;
            int live, tiles, blocks;
            x_extent<MODE>(s, at.b, live, tiles, blocks);
            if (tiles == 0 || blocks == 0) {  // no unit (never where a stretch starts or ends)
                ++at.b;
                continue;
            }
            const bool cut = at.b == to.b && at.h == to.h && at.p == to.p;
            const int end = cut ? to.blk : blocks;
            it.bh = at.b * s.Hkv + at.h;
            it.r0 = at.p * kXTile;
            it.b0 = at.blk;
            it.n_blk = end - at.blk;
            it.cols = MODE == kCrossDkv ? s.cols : live;
            it.live = live;
            it.reaches_end = end == blocks;
            it.part = at.blk == 0 && end == blocks ? -1 : 2 * cta + (pieces ? 1 : 0);
            ++pieces;
            if (cut) {
                at.blk = end;
            } else {
                at.blk = 0;
                if (++at.p == tiles) {
                    at.p = 0;
                    if (++at.h == s.Hkv) {
                        at.h = 0;
                        ++at.b;
                    }
                }
            }
            return true;
        }
        return false;
    }
};

// First row of a slot in the partial sums.
__device__ __forceinline__ long long x_part_row(const XSched &s, int part) {
    return (long long)part * s.slot_rows;
}

}  // namespace kata
