// sequence.h -- what the sequence operators (attention.hip, recurrence.hip) share:
// cutting jagged rows into tiles, and the edges of a segment.
#pragma once

#include "device.h"

namespace emb {

// The rows [0, n) of a jagged batch as segments 0 .. B + 1: segment j >= 1 is
// sample j - 1, and segments 0 and B + 1 are the rows before the first and after
// the last sample (usually none), which belong to nobody and read as empty.
// Offsets are clamped to [0, n], so no row outside the buffers is ever touched.
__device__ __forceinline__ int64_t seg_edge(const int32_t *off, int B, int64_t n, int64_t j)
{
    if (j <= 0) return 0;
    if (j >= B + 2) return n;
    const int64_t v = off[j - 1];
    return v < 0 ? 0 : v > n ? n : v;
}

// Tiles of `cut` rows that never cross a segment, found without a prefix sum over
// the segments: with e(j) the first row of segment j, its tiles are numbered from
// floor(e(j) / cut) + j.  floor(e(j+1) / cut) + 1 - floor(e(j) / cut) is at least
// ceil((e(j+1) - e(j)) / cut), so the numbers are enough; at most one or two a
// segment stay idle.  `mul` rows per offset unit (heads that share a key head are
// rows of their own).
__host__ __device__ __forceinline__ int64_t seg_tiles(int64_t n, int B, int mul, int cut)
{
    return n * mul / cut + B + 2;
}

struct SegTile {
    int64_t base;    // first row of the segment, in offset units
    int64_t row0;    // first row of the tile inside the segment (times mul)
    int64_t rows;    // rows of the segment (times mul); row0 >= rows: an idle tile
    int seg;         // segment number
};

// The segment of tile number `tile`, searched by the whole wavefront (64 probes a
// round): the last j with floor(e(j) * mul / cut) + j <= tile.
__device__ __forceinline__ SegTile seg_find(const int32_t *off, int B, int64_t n, int mul, int cut,
                                            int64_t tile)
{
    int64_t lo = 0, hi = B + 2;            // the answer is in [lo, hi)
    const int l = lane_id();
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 63) / 64;
        const int64_t j = lo + l * step;
        const bool le = j < hi && (j == lo || seg_edge(off, B, n, j) * mul / cut + j <= tile);
        const uint64_t m = __ballot(le);
        // probes that hold are a prefix of the lanes (lane 0 always holds)
        const int cnt = __popcll(m);
        const int64_t nlo = lo + (int64_t)(cnt - 1) * step;
        hi = nlo + step < hi ? nlo + step : hi;
        lo = nlo;
    }
    SegTile s;
    s.seg = uniform((int)lo);
    s.base = seg_edge(off, B, n, s.seg);
    const int64_t end = seg_edge(off, B, n, s.seg + 1);
    s.rows = end > s.base ? (end - s.base) * mul : 0;
    s.row0 = (tile - (s.base * mul / cut + s.seg)) * cut;
    if (s.row0 < 0) s.row0 = s.rows;       // offsets that decrease: nothing here
    return s;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint16_t bf16_rne(float x) { return (uint16_t)bf16x2_rne(x, 0.f); }

}  // namespace emb
