// sequence.h -- what the sequence operators (attention.hip, recurrence.hip) share:
// cutting jagged rows into tiles, and the edges of a segment.
#pragma once

#include "device.h"

namespace emb {

// Rows, keys, tiles and positions in them are 32-bit: the entry points refuse batches of more
// than kRowsMost rows (times the heads that share a key head).
constexpr int64_t kRowsMost = (int64_t(1) << 31) - 65536;

// The rows [0, n) of a jagged batch as segments 0 .. B + 1: segment j >= 1 is
// sample j - 1, and segments 0 and B + 1 are the rows before the first and after
// the last sample (usually none), which belong to nobody and read as empty.
// Offsets are clamped to [0, n], so no row outside the buffers is ever touched.
__device__ __forceinline__ int seg_edge(const int32_t *off, int B, int n, int j)
{
    const int at = j < 1 ? 0 : j > B + 1 ? B : j - 1;
    const int v = min(max(*gp(off + at), 0), n);
    return j < 1 ? 0 : j > B + 1 ? n : v;
}

// Tiles of `cut` rows that never cross a segment, found without a prefix sum over
// the segments: with e(j) the first row of segment j, its tiles are numbered from
// floor(e(j) / cut) + j.  floor(e(j+1) / cut) + 1 - floor(e(j) / cut) is at least
// ceil((e(j+1) - e(j)) / cut), so the numbers are enough; at most one or two a
// segment stay idle.  `mul` rows per offset unit (heads that share a key head are
// rows of their own).
inline int64_t seg_tiles(int64_t n, int B, int mul, int cut) { return n * mul / cut + B + 2; }

struct SegTile {
    int seg;         // segment number
    int base;        // first row of the segment, in offset units
    int row0;        // first row of the tile inside the segment (times mul)
    int rows;        // rows of the segment (times mul); row0 >= rows: an idle tile
    int o0, o1;      // the segment's rows on the other side (search with `other`)
};

// The segment of tile number `tile`, searched by the whole wavefront: the last j with
// floor(e(j) * mul / cut) + j <= tile.  64 probes a round; the last round, the only one
// up to 64 segments, reads both sides' edges along with the probes.
template <int cut>
__device__ __forceinline__ SegTile seg_find(const int32_t *off, int n, const int32_t *other, int no, int B, int mul,
                                            int tile)
{
    int lo = 0, hi = B + 2;            // the answer is in [lo, hi)
    const int l = lane_id();
    while (hi - lo > 64) {
        const int step = (hi - lo + 63) / 64, j = lo + l * step;
        const bool le = j < hi && (l == 0 || (int)((uint32_t)(seg_edge(off, B, n, j) * mul) / cut) + j <= tile);
        // probes that hold are a prefix of the lanes (lane 0 always holds)
        const int nlo = lo + (__popcll(__ballot(le)) - 1) * step;
        hi = min(nlo + step, hi);
        lo = nlo;
    }
    const int j = min(lo + l, hi - 1);
    const int e0 = seg_edge(off, B, n, j), e1 = seg_edge(off, B, n, j + 1);
    int p0 = 0, p1 = 0;
    if (other) {
        p0 = seg_edge(other, B, no, j);
        p1 = seg_edge(other, B, no, j + 1);
    }
    const bool le = lo + l < hi && (l == 0 || (int)((uint32_t)(e0 * mul) / cut) + j <= tile);
    const int at = __popcll(__ballot(le)) - 1;
    SegTile s;
    s.seg = uniform(lo + at);
    s.base = __builtin_amdgcn_readlane(e0, at);
    const int end = __builtin_amdgcn_readlane(e1, at);
    s.rows = end > s.base ? (end - s.base) * mul : 0;
    s.row0 = (tile - ((int)((uint32_t)(s.base * mul) / cut) + s.seg)) * cut;
    if (s.row0 < 0) s.row0 = s.rows;       // offsets that decrease: nothing here
    // rows of nobody have no other side
    const bool nobody = s.seg == 0 || s.seg == B + 1;
    s.o0 = nobody ? 0 : __builtin_amdgcn_readlane(p0, at);
    s.o1 = nobody ? 0 : max(__builtin_amdgcn_readlane(p1, at), s.o0);
    return s;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint16_t bf16_rne(float x) { return (uint16_t)bf16x2_rne(x, 0.f); }

}  // namespace emb
