// sequence.h -- what the sequence and encoder operators (attention.hip, recurrence.hip, delta.hip,
// norm.hip, rotary.hip) share: cutting jagged rows into tiles, the edges of a segment, LDS by
// address, rows in pieces of 16 bytes.
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

// ------------------------------------------------------ memory straight into LDS

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t lds_address(const void *p)
{
    return (uint32_t)uniform((int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p);
}

// LDS by its address as a number.
template <typename V>
__device__ __forceinline__ V lds_read(uint32_t at)
{
    return *(__attribute__((address_space(3))) const V *)(uintptr_t)at;
}

template <typename V>
__device__ __forceinline__ void lds_write(uint32_t at, V v)
{
    *(__attribute__((address_space(3))) V *)(uintptr_t)at = v;
}

// A 16-byte piece per lane from memory straight into 1 KB of LDS at `to`: lane l's
// piece lands at to + 16 l.  `off` counts bytes from the descriptor's base (plus the
// uniform `more`); an offset of kNowhere is out of the descriptor's range, reads no
// memory and lands as zeros.  The load is asynchronous (vmcnt): the compiler does not
// know of it, so the reader waits itself (arrived) before it reads.  Nor does it look for
// hazards in here: a scalar operand that a vector instruction wrote (readfirstlane, or a
// register spilled to lanes) may be read five wait states later, and the move and the
// s_nop are those five whatever came before.
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ void load_to_lds(i32x4_t rsrc, uint32_t to, uint32_t off, uint32_t more)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(to), "v"(off), "s"(rsrc), "s"(more)
                 : "memory");
}
// ... and before the tile it read from is overwritten, its LDS reads have to be done too
__device__ __forceinline__ void arrived() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ i32x4_t row_rsrc(const void *base)
{
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    i32x4_t r;
    r[0] = uniform((int)(uint32_t)b);
    r[1] = uniform((int)(uint32_t)(b >> 32) & 0xFFFF);
    r[2] = (int)kNowhere;
    r[3] = kBufFlags;
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint16_t bf16_rne(float x) { return (uint16_t)bf16x2_rne(x, 0.f); }

// 16 bytes of a row as numbers and back
template <typename T>
struct Piece;
template <>
struct Piece<uint16_t> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void open(const u32x4_t &w, float *f)
    {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            f[2 * j] = bf16_lo(w[j]);
            f[2 * j + 1] = bf16_hi(w[j]);
        }
    }
    static __device__ __forceinline__ u32x4_t shut(const float *f)
    {
        return u32x4_t{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7])};
    }
};
template <>
struct Piece<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void open(const u32x4_t &w, float *f)
    {
#pragma unroll
        for (int j = 0; j < 4; j++) f[j] = __uint_as_float(w[j]);
    }
    static __device__ __forceinline__ u32x4_t shut(const float *f)
    {
        return u32x4_t{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    }
};

}  // namespace emb
