// attention.hip -- cross attention of a sample's query rows over its key rows, both
// jagged, with a learned bias by buckets of the distance between their positions:
//   s_ij = scale q_i.k_j + bias[bucket(q_pos_i - k_pos_j), head],
//   p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
// and its backward pass
//   dP_ij = dO_i.v_j, delta_i = sum_j p_ij dP_ij, dS_ij = p_ij (dP_ij - delta_i),
//   dq_i = scale sum_j dS_ij k_j, dk_j = scale sum_i dS_ij q_i, dv_j = sum_i p_ij dO_i,
//   dbias[m] = sum of dS_ij over the pairs in bucket m.
//
// All products run on the matrix cores in 32 x 32 blocks, fp32 accumulators.  A
// block of scores comes out with one row (query) per lane & 31 and 16 of 32 keys in
// a lane's registers, register i of half h = lane >> 5 holding key
//   kk(i, h) = 8 (i >> 2) + 4 h + (i & 3).
// That is also the form in which the next product wants its second operand, if the
// keys of the contraction are taken in that order; so probabilities never leave the
// registers, and only the first operand (V, or K, Q, dO transposed) is read from LDS
// in the matching order, by the transposing LDS load for bf16.
//
// Times below were measured on one MI355X, bf16, at these sizes:
//   serving:  512 samples of 1..8 queries over 200..2000 keys, 4 heads of 64, 32 buckets
//   lifelong: 4 samples of 1 query over 60000..131072 keys, 8 heads on 2 of 128
//   many candidates: 32 samples of 100..500 queries over 200..2000 keys, 4 heads of 64, 32 buckets
//   ranking:  64 samples of 20..100 queries over 200..2000 keys, 4 heads of 64, 32 buckets
//   two sequences: 8 samples of 1500..2048 queries and keys, 8 heads of 128, 32 buckets
#include <algorithm>
#include <cmath>
#include <string>

#include "sequence.h"

namespace emb {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kBucketsMax = 256;
constexpr int kBiasWords = 4096;        // heads per key head x buckets held in LDS
constexpr int kAttnThreads = 256;
constexpr int kSplitsMax = 128;

struct AttnArgs {
    const void *q, *k, *v, *dout;
    int64_t qs, qh, ks, kh, vs, vh, ds, dh;     // row and head strides in elements
    const int32_t *qo, *ko;                     // [samples + 1]
    const uint8_t *mask;                        // [n_k] or NULL
    const int32_t *qp, *kp, *bnd;               // positions, boundaries [buckets - 1]
    const float *bias;                          // [buckets, heads] or NULL
    int32_t nq, nk;
    int32_t samples, heads, kv_heads, group, dim, buckets;
    float scale, rscale, c;                     // rscale = 1 / scale, c = scale * log2(e)
    int32_t vec, ovec, gvec;                    // rows (of out, of dk and dv) move in 16-byte pieces
    int32_t splits, chunk;
    int32_t tiles;
    void *out, *rest;                           // [n_q, heads, dim]; what rounding out left, or NULL
    float *lse;                                 // [n_q, heads]
    float *part, *part_ml;                      // split partials
    void *dq, *dk, *dv;
    float *delta;                               // [n_q, heads]
    float *dbias_part;                          // [tiles, heads, buckets]
};

__device__ __forceinline__ int sub_sat(int a, int b) { return __builtin_elementwise_sub_sat(a, b); }

// ------------------------------------------------------------- tiles in LDS

// A tile holds rows of DP elements (the head size padded with zeros) in 16-byte
// chunks; chunk c of row r sits at place c ^ swizzle(r), so that both 16 lanes that
// read one chunk of 16 consecutive rows and 32 lanes that read 4 chunks of 4
// consecutive rows touch all 64 banks once.
template <int CH>
__device__ __forceinline__ int swizzle(int r)
{
    if (CH == 4) return (r >> 2) & 3;
    if (CH == 8) return ((r & 2) << 1) | ((r >> 2) & 3);
    return ((r & 3) << 2) | ((r >> 2) & 3);
}

template <typename T, int DP>
struct Tile {
    static constexpr int E = 16 / sizeof(T);         // elements per chunk
    static constexpr int CH = DP / E;                // chunks per row
    static __device__ __forceinline__ int at(int r, int c) { return r * CH + (c ^ swizzle<CH>(r)); }
};

// The products below read tiles by LDS address (lds_read): the lane's part is one number, and chunk
// and row of a read come in as a constant xor and a constant offset (the swizzle is a xor of row
// bits, and tiles are aligned to a row).  So a read costs one xor and no register that outlives it.

// a row as a second operand: its even chunks in half 0, its odd ones in half 1
template <typename T, int DP>
using Frag = u32x4_t[Tile<T, DP>::CH / 2];

// one 16-byte chunk of a row in memory; elements past `dim` read as zero
template <typename T>
__device__ __forceinline__ u32x4_t load_chunk(const T *row, int c, int dim, bool vec)
{
    constexpr int E = 16 / sizeof(T);
    u32x4_t z = {0, 0, 0, 0};
    if (c * E >= dim) return z;
    if (vec) return *gp(reinterpret_cast<const u32x4_t *>(row + c * E));
    union {
        u32x4_t w;
        T e[E];
    } u;
    u.w = z;
#pragma unroll
    for (int i = 0; i < E; i++)
        if (c * E + i < dim) u.e[i] = *gp(row + c * E + i);
    return u.w;
}

// ------------------------------------------------------------ matrix products

template <typename T>
struct Mma;

template <>
struct Mma<uint16_t> {
    // acc += A B over 16 elements of the contraction: lane & 31 is A's row and B's
    // column, half h = lane >> 5 holds elements 8 h .. 8 h + 7 in one chunk
    static __device__ __forceinline__ void chunk(f32x16_t &acc, u32x4_t a, u32x4_t b)
    {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                      __builtin_bit_cast(bf16x8_t, b), acc, 0, 0, 0);
    }
    // a 32 x 32 block of weights (row or key per lane) as second operands, bf16
    struct Pack {
        u32x4_t w[2];
    };
    static __device__ __forceinline__ Pack pack(const f32x16_t &p)
    {
        Pack r;
#pragma unroll
        for (int kc = 0; kc < 2; kc++)
#pragma unroll
            for (int j = 0; j < 4; j++) r.w[kc][j] = bf16x2_rne(p[8 * kc + 2 * j], p[8 * kc + 2 * j + 1]);
        return r;
    }
    // 32 rows of a tile from r0 (a multiple of 32), elements 32 db .. of each, transposed, as
    // first operand: times(): acc[d, lane] += sum over the 32 rows of tile[row, d] w[row, lane]
    template <int DP>
    struct Rows {
        s16x8_t a[2];
        __device__ __forceinline__ Rows(const u32x4_t *tile, int r0, int db)
        {
            using TL = Tile<uint16_t, DP>;
            // sixteen lanes read 4 rows of 16 elements and get a column of 4 each
            const int l = lane_id(), row = 4 * (l >> 5) + ((l & 15) >> 2), col = 16 * ((l >> 4) & 1) + 4 * (l & 3);
            const uint32_t base = lds_address(tile) + 16 * TL::at(row, col >> 3) + (col & 7) * 2;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int kc = j >> 1, jb = j & 1;
                const uint32_t at = (base ^ ((4 * db) ^ swizzle<TL::CH>(8 * jb)) << 4) + (r0 + 16 * kc + 8 * jb) * TL::CH * 16;
                const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4_t *)(uintptr_t)at);
#pragma unroll
                for (int e = 0; e < 4; e++) a[kc][4 * jb + e] = v[e];
            }
        }
        __device__ __forceinline__ void times(f32x16_t &acc, const Pack &w) const
        {
#pragma unroll
            for (int kc = 0; kc < 2; kc++)
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a[kc]),
                                                              __builtin_bit_cast(bf16x8_t, w.w[kc]), acc, 0, 0, 0);
        }
    };
    static __device__ __forceinline__ float dot(u32x4_t a, u32x4_t b)
    {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 4; j++) s += bf16_lo(a[j]) * bf16_lo(b[j]) + bf16_hi(a[j]) * bf16_hi(b[j]);
        return s;
    }
    static __device__ __forceinline__ u32x2_t pack4(const float *v)
    {
        return u32x2_t{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
    }
    static __device__ __forceinline__ void store4(uint16_t *p, const float *v)
    {
        *gp(reinterpret_cast<u32x2_t *>(p)) = pack4(v);
    }
    static __device__ __forceinline__ void store1(uint16_t *p, float v) { *gp(p) = bf16_rne(v); }
};

template <>
struct Mma<float> {
    static __device__ __forceinline__ void chunk(f32x16_t &acc, u32x4_t a, u32x4_t b)
    {
#pragma unroll
        for (int j = 0; j < 4; j++)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[j]), __uint_as_float(b[j]), acc, 0, 0, 0);
    }
    struct Pack {
        f32x16_t w;
    };
    static __device__ __forceinline__ Pack pack(const f32x16_t &p) { return Pack{p}; }
    template <int DP>
    struct Rows {
        f32x16_t a;
        __device__ __forceinline__ Rows(const u32x4_t *tile, int r0, int db)
        {
            using TL = Tile<float, DP>;
            const int l = lane_id(), h = l >> 5, d = l & 31;
            const uint32_t base = lds_address(tile) + 16 * TL::at(4 * h, d >> 2) + (d & 3) * 4;
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const int row = 8 * (i >> 2) + (i & 3);
                a[i] = lds_read<float>((base ^ ((8 * db) ^ swizzle<TL::CH>(row)) << 4) + (r0 + row) * TL::CH * 16);
            }
        }
        __device__ __forceinline__ void times(f32x16_t &acc, const Pack &w) const
        {
#pragma unroll
            for (int i = 0; i < 16; i++) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], w.w[i], acc, 0, 0, 0);
        }
    };
    static __device__ __forceinline__ float dot(u32x4_t a, u32x4_t b)
    {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 4; j++) s = fmaf(__uint_as_float(a[j]), __uint_as_float(b[j]), s);
        return s;
    }
    static __device__ __forceinline__ f32x4_t pack4(const float *v) { return f32x4_t{v[0], v[1], v[2], v[3]}; }
    static __device__ __forceinline__ void store4(float *p, const float *v)
    {
        *gp(reinterpret_cast<f32x4_t *>(p)) = pack4(v);
    }
    static __device__ __forceinline__ void store1(float *p, float v) { *gp(p) = v; }
};

// acc += (32 rows of a tile) x (32 rows held as second operands): the block of
// scalar products of two sets of DP-element rows
template <typename T, int DP>
__device__ __forceinline__ void products(f32x16_t &acc, const u32x4_t *tile, int r0,
                                         const Frag<T, DP> &b)
{
    using TL = Tile<T, DP>;
    const int l = lane_id();
    const uint32_t base = lds_address(tile + r0 * TL::CH) + 16 * TL::at(l & 31, l >> 5);
#pragma unroll
    for (int c = 0; c < TL::CH / 2; c++) Mma<T>::chunk(acc, lds_read<u32x4_t>(base ^ (c << 5)), b[c]);
}

// The same with the second operands' rows in a tile too: twice the LDS reads, but none
// of the registers.
template <typename T, int DP>
__device__ __forceinline__ void products(f32x16_t &acc, const u32x4_t *tile, int r0, const u32x4_t *other, int o0)
{
    using TL = Tile<T, DP>;
    const int l = lane_id();
    const uint32_t mine = 16 * TL::at(l & 31, l >> 5);
    const uint32_t a = lds_address(tile + r0 * TL::CH) + mine, b = lds_address(other + o0 * TL::CH) + mine;
#pragma unroll
    for (int c = 0; c < TL::CH / 2; c++)
        Mma<T>::chunk(acc, lds_read<u32x4_t>(a ^ (c << 5)), lds_read<u32x4_t>(b ^ (c << 5)));
}

// 16 values of a 32-entry array in the order of a block's registers
__device__ __forceinline__ f32x16_t block_order(const float *v)
{
    const int h = lane_id() >> 5;
    f32x16_t r;
#pragma unroll
    for (int g = 0; g < 4; g++) {
        const float4 w = *reinterpret_cast<const float4 *>(v + 8 * g + 4 * h);
        r[4 * g] = w.x;
        r[4 * g + 1] = w.y;
        r[4 * g + 2] = w.z;
        r[4 * g + 3] = w.w;
    }
    return r;
}
__device__ __forceinline__ int block_key(int i) { return 8 * (i >> 2) + 4 * (lane_id() >> 5) + (i & 3); }

// x combined with the other half's value of the same lane & 31
__device__ __forceinline__ float both_halves_max(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float both_halves_sum(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum over the wavefront, minimum and maximum over 32 lanes, with DPP moves: inside
// quads, half rows, rows of 16, then the last lane of a row into the next.
#define EMB_DPP(x, ctrl, rows) __builtin_amdgcn_update_dpp(x, x, ctrl, rows, 0xF, false)
__device__ __forceinline__ float wave_sum(float x)
{
    auto add = [](float v, int moved) { return v + __int_as_float(moved); };
    x = add(x, EMB_DPP(__float_as_int(x), 0xB1, 0xF));
    x = add(x, EMB_DPP(__float_as_int(x), 0x4E, 0xF));
    x = add(x, EMB_DPP(__float_as_int(x), 0x141, 0xF));
    x = add(x, EMB_DPP(__float_as_int(x), 0x140, 0xF));
    // every lane now holds its row's sum
    float r = 0.f;
#pragma unroll
    for (int l = 15; l < 64; l += 16) r += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), l));
    return r;
}
struct Range {
    int lo, hi;
};
// of the 32 values of half u: the ends where they are in order, as positions mostly are
__device__ __forceinline__ Range half_range(int x, int u = 0)
{
    const int before = EMB_DPP(x, 0x138, 0xF);      // wave_shr:1, lane 0 keeps its own
    if (((uint32_t)(__ballot(before <= x) >> (32 * u)) | 1) == 0xFFFFFFFFu)
        return Range{__builtin_amdgcn_readlane(x, 32 * u), __builtin_amdgcn_readlane(x, 32 * u + 31)};
    int a = x, b = x;
    a = min(a, EMB_DPP(a, 0xB1, 0xF));
    b = max(b, EMB_DPP(b, 0xB1, 0xF));
    a = min(a, EMB_DPP(a, 0x4E, 0xF));
    b = max(b, EMB_DPP(b, 0x4E, 0xF));
    a = min(a, EMB_DPP(a, 0x141, 0xF));
    b = max(b, EMB_DPP(b, 0x141, 0xF));
    a = min(a, EMB_DPP(a, 0x140, 0xF));
    b = max(b, EMB_DPP(b, 0x140, 0xF));
    return Range{min(__builtin_amdgcn_readlane(a, 32 * u), __builtin_amdgcn_readlane(a, 32 * u + 16)),
                 max(__builtin_amdgcn_readlane(b, 32 * u), __builtin_amdgcn_readlane(b, 32 * u + 16))};
}
#undef EMB_DPP

// ------------------------------------------------------------------ the bias

// The bias table of a key head's group, over scale, and the boundaries, in LDS: so an
// entry can be where a block of products starts, and the scaling brings it back.  Finite
// entries are held to +-kBiasMost, where fp32 still tells scores apart that differ by a
// hundredth; a weight of e^-kBiasMost beside any other is zero.  The boundaries also in
// registers, one or more a lane, so that the bucket of a uniform distance is a count over
// ballots.  Loads are issued first (take) and used later (put): nothing they need depends
// on the offsets.
constexpr float kBiasMost = 1e5f;
struct Bias {
    int b[kBucketsMax / 64];
    int n;               // boundaries
    float first;         // this thread's first entry of the table

    static __device__ __forceinline__ int64_t entry(const AttnArgs &A, int kvh, int i)
    {
        const int m = i / A.group, g = i - m * A.group;
        return (int64_t)m * A.heads + kvh * A.group + g;
    }
    __device__ __forceinline__ void take(const AttnArgs &A, int kvh)
    {
        n = A.bias ? A.buckets - 1 : 0;
        first = 0.f;
#pragma unroll
        for (int t = 0; t < kBucketsMax / 64; t++) {
            const int j = 64 * t + lane_id();
            b[t] = j < n ? *gp(A.bnd + j) : INT32_MAX;
        }
        if ((int)threadIdx.x < A.buckets * A.group) first = *gp(A.bias + entry(A, kvh, threadIdx.x));
    }
    __device__ __forceinline__ void put(const AttnArgs &A, int kvh, float *lb, int *lbnd) const
    {
        if (!A.bias) return;
        const int t = threadIdx.x, all = A.buckets * A.group;
        auto held = [&](float x) {
            return fabsf(x) > kBiasMost && fabsf(x) < INFINITY ? copysignf(kBiasMost, x) * A.rscale : x * A.rscale;
        };
        if (t < all) lb[t] = held(first);
        for (int i = t + kAttnThreads; i < all; i += kAttnThreads) lb[i] = held(*gp(A.bias + entry(A, kvh, i)));
        if (t < 64)
#pragma unroll
            for (int u = 0; u < kBucketsMax / 64; u++)
                if (64 * u + t < n) lbnd[64 * u + t] = b[u];
    }
    __device__ __forceinline__ int bucket(int x) const
    {
        int c = 0;
#pragma unroll
        for (int t = 0; t < kBucketsMax / 64; t++)
            if (64 * t < n) c += __popcll(__ballot(b[t] <= x));
        return uniform(min(c, n));
    }
};

// The bucket that the last blocks of scores fell into whole, as the range of distances
// it covers.  Neighbouring blocks mostly share a bucket (buckets widen with the
// distance), and then two compares a block say so.
struct BucketRun {
    int m, lo, last;     // bucket, and its distances lo .. last

    __device__ __forceinline__ void set(const Bias &B, const int *lbnd, int bucket)
    {
        m = bucket;
        lo = m > 0 ? lbnd[m - 1] : INT32_MIN;
        last = m < B.n ? lbnd[m] - 1 : INT32_MAX;     // a bucket in use ends above INT32_MIN
    }
    // lanes whose distances a .. b all lie in the bucket
    __device__ __forceinline__ uint64_t covers(int a, int b) const { return __ballot(a >= lo && b <= last); }
};

// ------------------------------------------------------ rows into LDS tiles

// Brings ROWS rows (of `rows` that begin at element pointer `base`, `stride` elements
// apart) into a tile's rows r0 .., by one wavefront; row r whose bit in `keep` is clear
// becomes zeros and is not read.  Masked rows have to be zeros: a probability of zero
// must not meet an infinity or NaN.
template <typename T, int DP, int ROWS>
__device__ __forceinline__ void bring_rows(const T *base, int64_t stride, int dim, bool vec, uint64_t keep,
                                           u32x4_t *tile, int r0)
{
    using TL = Tile<T, DP>;
    constexpr int PER = 64 / TL::CH;                    // rows per load
    const int l = lane_id(), rl = l / TL::CH;
    const int c0 = (l % TL::CH) ^ swizzle<TL::CH>(rl);  // swizzle is a xor of row bits
    u32x4_t *to = tile + r0 * TL::CH;
    if (vec) {
        const i32x4_t rsrc = row_rsrc(base);
        const uint32_t lds = lds_address(to), mine = (uint32_t)(rl * (int)stride) * sizeof(T);
        const uint64_t bits = keep >> rl;
#pragma unroll
        for (int j = 0; j < ROWS / PER; j++) {
            const int c = c0 ^ swizzle<TL::CH>((r0 + j * PER) & 15);
            const bool in = (bits >> (j * PER) & 1) && c * TL::E < dim;
            load_to_lds(rsrc, lds + j * 1024, in ? mine + c * 16 : kNowhere,
                        (uint32_t)(j * PER * (int)stride) * sizeof(T));
        }
        return;
    }
#pragma unroll 2
    for (int j = 0; j < ROWS / PER; j++) {
        const int r = j * PER + rl, c = c0 ^ swizzle<TL::CH>((r0 + j * PER) & 15);
        u32x4_t v = {0, 0, 0, 0};
        if (keep >> r & 1) v = load_chunk(base + r * stride, c, dim, false);
        to[j * 64 + l] = v;
    }
}

// What a workgroup does: tiles of one key head are neighbours in the order of work, and
// pieces of `chunk` of that order go to the XCDs in turn.
struct Task {
    int split, kvh, tile;
};
__device__ __forceinline__ Task task(const AttnArgs &A)
{
    const uint32_t id = (uint32_t)xcd_block(blockIdx.x, gridDim.x, A.chunk), rest = id / (uint32_t)A.splits;
    Task t;
    t.split = (int)(id - rest * (uint32_t)A.splits);
    t.kvh = (int)(rest / (uint32_t)A.tiles);
    t.tile = (int)(rest - (uint32_t)t.kvh * (uint32_t)A.tiles);
    return t;
}

// The range of pieces a split takes of `n`.
__device__ __forceinline__ void split_range(int n, int split, int splits, int &a, int &b)
{
    a = (int)((uint64_t)n * split / (uint32_t)splits);
    b = (int)((uint64_t)n * (split + 1) / (uint32_t)splits);
    if (splits == 1) a = 0, b = n;
}

// The 32 query rows of a wavefront, one per lane & 31 (both halves hold the same).
struct Row {
    bool live;
    int q;           // row of q
    int head, g;     // query head, its number inside the group
    int pos;
    Range r;         // of positions of the wavefront's rows

    __device__ __forceinline__ void range() { r = half_range(pos); }
};

__device__ __forceinline__ Row query_row(const AttnArgs &A, const SegTile &s, int kvh, int r0)
{
    Row R;
    const int r = r0 + (lane_id() & 31);
    R.live = r < s.rows;
    const uint32_t rc = R.live ? r : s.rows - 1;     // a row past the end repeats the last
    const uint32_t i = A.group == 1 ? rc : rc / (uint32_t)A.group;
    R.g = (int)(rc - i * A.group);
    R.q = s.base + i;
    R.head = kvh * A.group + R.g;
    R.pos = A.bias ? *gp(A.qp + R.q) : 0;
    return R;
}

template <typename T, int DP>
__device__ __forceinline__ void load_frag(Frag<T, DP> &f, const T *row, int dim, bool vec, bool live)
{
    const int h = lane_id() >> 5;
#pragma unroll
    for (int c = 0; c < Tile<T, DP>::CH / 2; c++) {
        const u32x4_t z = {0, 0, 0, 0};
        f[c] = live ? load_chunk(row, 2 * c + h, dim, vec) : z;
    }
}

// Whether a block of products starts from its bias or gets it added.  bf16 products of a
// head are 2 to 8 accumulations and the start costs nothing; fp32 products are four times
// as many, and rounding each at the bias's size would cost the gradients a digit (error of
// an fp32 dbias against 64 bits: 2.2e-6 with the bias first, 4.3e-7 with it added).
template <typename T>
constexpr bool kBiasFirst = sizeof(T) == 2;

// Scores in units of log2 are t_i = c s_i + b with s_i the product (plus what the block
// started from) and b a number per row: where all pairs of a block fall in one bucket the
// bias is in b and costs nothing.  Where they do not, each boundary inside the block's
// range is a compare and a select on what the block starts from, and b is zero.  This
// is for blocks outside the bucket of `run`: afterwards `run` is the bucket of the
// block's smallest distance and b_run its bias.
// `kpos`: positions of the tile's keys in LDS, `pos`: the same, one a lane; u: which 32;
// all: no key of the block is at -inf already.
// Everything that comes out of LDS is asked for together: the latency of this is what a
// mixed block costs.
template <typename T>
__device__ __forceinline__ void mixed_bias(const AttnArgs &A, const Bias &B, const float *lb, const int *lbnd,
                                           const Row &R, const int *kpos, int pos, int u, bool all,
                                           BucketRun &run, f32x16_t &s, float &b, float &b_run)
{
    const int h = lane_id() >> 5;
    int4 k4[4];
#pragma unroll
    for (int g = 0; g < 4; g++) k4[g] = *reinterpret_cast<const int4 *>(kpos + 32 * u + 8 * g + 4 * h);
    const Range k = half_range(pos, u);
    const int lo = B.bucket(sub_sat(R.r.lo, k.hi)), hi = B.bucket(sub_sat(R.r.hi, k.lo));
    const float *mine = lb + R.g;
    const float base = mine[lo * A.group];
    float v = mine[min(lo + 1, hi) * A.group];
    int edge = lbnd[lo];                 // not read for the last bucket
    run.set(B, lbnd, lo);
    b = b_run = base * A.c;
    if (lo == hi) return;
    b = 0.f;
    int x[16];
#pragma unroll
    for (int g = 0; g < 4; g++) {
        x[4 * g] = sub_sat(R.pos, k4[g].x);
        x[4 * g + 1] = sub_sat(R.pos, k4[g].y);
        x[4 * g + 2] = sub_sat(R.pos, k4[g].z);
        x[4 * g + 3] = sub_sat(R.pos, k4[g].w);
    }
    f32x16_t t;
#pragma unroll
    for (int i = 0; i < 16; i++) t[i] = x[i] >= edge ? v : base;
    for (int m = lo + 1; m < hi; m++) {
        edge = lbnd[m];
        v = mine[(m + 1) * A.group];
#pragma unroll
        for (int i = 0; i < 16; i++) t[i] = x[i] >= edge ? v : t[i];
    }
    // s holds 0 or products, or -inf where a key takes no part: there whatever t holds, an
    // infinity or NaN too
    const f32x16_t with = kBiasFirst<T> ? t : s + t;
    if (all) {
        s = with;
    } else {
#pragma unroll
        for (int i = 0; i < 16; i++) s[i] = s[i] == -INFINITY ? s[i] : with[i];
    }
}

// What the kernels that walk the keys share.  WM = 4: the four wavefronts take 32 query
// rows each, share tiles of KT keys, and meet at a barrier per tile.  WM = 1 (few rows
// per sample): all take the same 32 rows; each walks every fourth 32 keys with tiles of
// its own and no barrier, and the four results meet at the end.  Either way the next
// tile is on its way into the other buffer while one is worked on (kBufs = 2, where
// two fit into LDS).
template <typename T, int DP, int WM>
struct KeyWalk {
    using TL = Tile<T, DP>;
    static constexpr int KT = WM == 4 && sizeof(T) == 2 ? 64 : 32;
    static constexpr int kOwners = WM == 4 ? 1 : 4;             // sets of tiles
    static constexpr int kWords = KT * TL::CH;                  // of K or V, 16 bytes each
    static constexpr int kBufs = kOwners * 4 * kWords * 16 <= 131072 ? 2 : 1;
    static constexpr int kLds = kOwners * kBufs * 2 * kWords;
    // Wavefronts per SIMD to build for: two wherever LDS lets two workgroups on
    // a CU.  That also caps a wavefront at 256 registers, and then the compiler keeps the
    // accumulators where the rescaling can use them; with the full 512 it puts them in the
    // other half of the file and moves each of them back and forth in every step (2048-row
    // sequences, 8 heads of 128: 321 us, against 186 us).
    static constexpr int kWaves = kLds * 16 <= 72 * 1024 && !(sizeof(T) == 4 && DP == 128) ? 2 : 1;
    static_assert(KT / (WM == 4 ? 4 : 1) >= 64 / TL::CH, "a load covers whole rows of one wavefront's share");

    static constexpr int kStep = WM == 1 ? 4 : 1;
    static constexpr int R = WM == 4 ? KT / 4 : KT;     // rows of a tile that a wavefront brings

    u32x4_t *mine;           // this wavefront's tiles
    const AttnArgs &A;
    int w, buf;
    int at, end;             // tiles [at, end) of KT keys to go
    const T *k, *v;          // rows to bring next
    int look_key, k1;    // key to look at next; end of the sample
    uint64_t keep;           // keys of the current tile that take part
    int pos;                 // position of the current tile's key lane (KT = 64) or lane & 31
    uint64_t keep_next;      // of the tile after the current one
    int pos_next;
    int raw_keep, raw_pos;   // loads in flight for the tile after that

    __device__ __forceinline__ KeyWalk(const AttnArgs &a, u32x4_t *lds, int kvh, int w_, int k0, int k1_, int split)
        : A(a), w(w_), buf(0), k1(k1_), raw_pos(0)
    {
        mine = lds + (WM == 4 ? 0 : w * (kLds / 4));
        split_range(k1 > k0 ? (k1 - k0 + KT - 1) / KT : 0, split, A.splits, at, end);
        if (WM == 1) at += w;
        const int key = k0 + at * KT;
        const int64_t row = key + (WM == 4 ? w * R : 0);
        look_key = key + (lane_id() & (KT - 1));
        k = static_cast<const T *>(A.k) + kvh * A.kh + row * A.ks;
        v = static_cast<const T *>(A.v) + kvh * A.vh + row * A.vs;
    }

    __device__ __forceinline__ const u32x4_t *k_tile() const { return mine + buf * 2 * kWords; }
    __device__ __forceinline__ const u32x4_t *v_tile() const { return mine + buf * 2 * kWords + kWords; }

    // mask and position of the keys of a tile, one key a lane; past the sample's end
    // the last key is looked at again
    __device__ __forceinline__ void look()
    {
        const bool in = look_key < k1;
        const int key = in ? look_key : k1 - 1;
        raw_keep = in ? (A.mask ? *gp(A.mask + key) : 1) : 0;
        if (A.bias) raw_pos = *gp(A.kp + key);
        look_key += kStep * KT;
    }
    __device__ __forceinline__ void seen()
    {
        keep_next = __ballot(raw_keep != 0);
        if (KT == 32) keep_next &= 0xFFFFFFFFull;
        pos_next = raw_pos;
    }
    __device__ __forceinline__ void bring(int to)
    {
        u32x4_t *lk = mine + to * 2 * kWords, *lv = lk + kWords;
        const int r0 = WM == 4 ? w * R : 0;
        bring_rows<T, DP, R>(k, A.ks, A.dim, A.vec, keep_next >> r0, lk, r0);
        bring_rows<T, DP, R>(v, A.vs, A.dim, A.vec, keep_next >> r0, lv, r0);
        k += kStep * KT * A.ks;
        v += kStep * KT * A.vs;
    }
    __device__ __forceinline__ void start()
    {
        if (at >= end) return;
        look();
        seen();
        if (kBufs == 2) bring(0);
        look();
    }
    // the current tile is in LDS after this, and the next on its way
    __device__ __forceinline__ void enter()
    {
        keep = keep_next;
        pos = pos_next;
        if (kBufs == 1) {
            arrived();
            if (WM == 4) __syncthreads();
            bring(0);
        }
        arrived();
        if (WM == 4) __syncthreads();
        else wave_sync();
        seen();
        if (kBufs == 2 && at + kStep < end) bring(buf ^ 1);
        look();
    }
    __device__ __forceinline__ void leave()
    {
        at += kStep;
        if (kBufs == 2) buf ^= 1;
    }
};

// The four wavefronts' blocks x (DP elements of 32 rows each) summed through LDS;
// wavefront w gets elements 32 d + 8 w + 4 h + e of row lane & 31 in r[d][e].
template <int DP>
__device__ __forceinline__ void sum_waves(float *lds, const f32x16_t (&x)[DP / 32], int w, float (&r)[DP / 32][4])
{
    const int lane = lane_id(), h = lane >> 5;
#pragma unroll
    for (int d = 0; d < DP / 32; d++) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; i++) lds[(w * 32 + block_key(i)) * 32 + (lane & 31)] = x[d][i];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; e++) {
            float z = 0.f;
#pragma unroll
            for (int u = 0; u < 4; u++) z += lds[(u * 32 + 8 * w + 4 * h + e) * 32 + (lane & 31)];
            r[d][e] = z;
        }
    }
}

template <typename T>
__device__ __forceinline__ void store_part(T *row, int col, int dim, const float *v)
{
    if (col + 4 <= dim && dim % 4 == 0) Mma<T>::store4(row + col, v);
    else
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (col + e < dim) Mma<T>::store1(row + col + e, v[e]);
}

// ... of the output, with what the rounding leaves of each element beside it
template <typename T>
__device__ __forceinline__ void store_out(const AttnArgs &A, int64_t row, int col, const float *v)
{
    store_part(static_cast<T *>(A.out) + row * A.dim, col, A.dim, v);
    if (sizeof(T) == 4 || !A.rest) return;
    float r[4];
#pragma unroll
    for (int e = 0; e < 4; e++) r[e] = v[e] - bf16_lo(bf16_rne(v[e]));
    store_part(static_cast<T *>(A.rest) + row * A.dim, col, A.dim, r);
}

// 1 / l, zero for a row without keys; NaN stays
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float log_sum(float m, float l)
{
    return l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// ------------------------------------------------------------------ forward

// The running maximum m of a row may lag behind by 2^kLag: the weights stay far from
// overflow, and the accumulators are rescaled only when it has to move.
constexpr float kLag = 8.f;

// One pass over the keys with the running maximum and sum of the softmax; scores and
// weights stay in registers.  The weights enter their product in T, as the values do: a
// relative error of up to 2^-8 each, independent ones, where the output's own rounding
// is as large; their sum l is of the fp32 weights.
// Serving 122 us (4.7 TB/s of its 576 MB) and lifelong 85 us and 5 us for the join (4.5
// TB/s of 408 MB), where a large copy has 5.5: the reading bounds them.  Two sequences
// 218 us, 458 TFLOP/s (without a bias 156): two wavefronts a SIMD alternate between
// products and weights, and the blocks whose pairs fall into several buckets cost the
// rest.  Many candidates 62 us, 151 TFLOP/s (without a bias 49): a workgroup has 9 steps
// between its first loads (four dependent ones) and its join, and these do not overlap.
template <typename T, int DP, int WM>
__global__ __launch_bounds__(kAttnThreads, (KeyWalk<T, DP, WM>::kWaves)) void attn_forward(AttnArgs A)
{
    using KW = KeyWalk<T, DP, WM>;
    constexpr int SUBS = KW::KT / 32;
    __shared__ __align__(1024) u32x4_t lds[KW::kLds > 1024 ? KW::kLds : 1024];    // 16 KB for sum_waves
    __shared__ int lbnd[kBucketsMax];
    __shared__ __align__(16) int kpos[4][32 * SUBS];
    __shared__ __align__(16) float kout[4][32];
    __shared__ float jm[4][32], jl[4][32];
    extern __shared__ float lb[];

    const Task job = task(A);
    const int split = job.split, kvh = job.kvh;
    if (kvh >= A.kv_heads) return;
    Bias B;
    B.take(A, kvh);
    const SegTile s = seg_find<WM * 32>(A.qo, A.nq, A.ko, A.nk, A.samples, A.group, job.tile);
    if (s.row0 >= s.rows) return;
    const int lane = lane_id(), h = lane >> 5, w = uniform((int)(threadIdx.x >> 6));
    const int r0 = s.row0 + (WM == 4 ? w * 32 : 0);
    const bool busy = r0 < s.rows;

    Row R = query_row(A, s, kvh, r0);
    Frag<T, DP> qf;
    load_frag<T, DP>(qf, static_cast<const T *>(A.q) + (int64_t)R.q * A.qs + R.head * A.qh, A.dim, A.vec, R.live);
    KW walk(A, lds, kvh, w, s.o0, s.o1, split);
    walk.start();
    B.put(A, kvh, lb, lbnd);
    R.range();
    if (A.bias) __syncthreads();      // the bias table
    BucketRun run{0, INT32_MAX, INT32_MIN};
    float b_run = 0.f;
    if (A.bias && walk.at < walk.end) {
        // the first keys' bucket, while they are on their way
        run.set(B, lbnd, B.bucket(sub_sat(R.r.lo, half_range(walk.pos_next).hi)));
        b_run = lb[run.m * A.group + R.g] * A.c;
    }

    float m = -INFINITY, l = 0.f;
    f32x16_t o[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; d++) o[d] = f32x16_t{};

    for (; walk.at < walk.end; walk.leave()) {
        walk.enter();
        if (!busy || walk.keep == 0) continue;
        const u32x4_t *lk = walk.k_tile(), *lv = walk.v_tile();
        f32x16_t sc[SUBS];
        float b[SUBS], top = -INFINITY;
        uint64_t in_run = A.bias ? run.covers(sub_sat(R.r.lo, walk.pos), sub_sat(R.r.hi, walk.pos)) : ~0ull;
        if (~in_run) {
            kpos[w][lane & (32 * SUBS - 1)] = walk.pos;
            wave_sync();
        }
#pragma unroll
        for (int u = 0; u < SUBS; u++) {
            const uint32_t keep = (uint32_t)(walk.keep >> (32 * u));
            sc[u] = f32x16_t{};
            if (keep != 0xFFFFFFFFu) {
                // keys that take no part start at -inf (their K is zero)
                kout[w][lane & 31] = keep >> (lane & 31) & 1 ? 0.f : -INFINITY;
                wave_sync();
                sc[u] = block_order(kout[w]);
                wave_sync();
            }
            b[u] = b_run;
            if (!kBiasFirst<T>) products<T, DP>(sc[u], lk, u * 32, qf);
            if (~in_run >> (32 * u) & 0xFFFFFFFFu) {
                mixed_bias<T>(A, B, lb, lbnd, R, kpos[w], walk.pos, u, keep == 0xFFFFFFFFu, run, sc[u], b[u],
                              b_run);
                if (u + 1 < SUBS) in_run = run.covers(sub_sat(R.r.lo, walk.pos), sub_sat(R.r.hi, walk.pos));
            }
            b[u] = keep ? b[u] : 0.f;         // a bias that only masked keys have
            if (kBiasFirst<T>) products<T, DP>(sc[u], lk, u * 32, qf);
        }
#pragma unroll
        for (int u = 0; u < SUBS; u++) {
            float t = sc[u][0];
#pragma unroll
            for (int i = 1; i < 16; i++) t = fmaxf(t, sc[u][i]);
            top = fmaxf(top, fmaf(t, A.c, b[u]));
        }
        top = both_halves_max(top);
        if (__ballot(top > m + kLag)) {
            const float mn = fmaxf(m, top);
            const float alpha = exp2_fast(m - (mn == -INFINITY ? 0.f : mn));
            m = mn;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < DP / 32; d++)
#pragma unroll
                for (int i = 0; i < 16; i++) o[d][i] *= alpha;
        }
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int u = 0; u < SUBS; u++) {
            const float bu = b[u] - base;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 16; i++) {
                sc[u][i] = exp2_fast(fmaf(sc[u][i], A.c, bu));
                sum += sc[u][i];
            }
            l += sum;
            const typename Mma<T>::Pack p = Mma<T>::pack(sc[u]);
#pragma unroll
            for (int d = 0; d < DP / 32; d++) typename Mma<T>::template Rows<DP>(lv, u * 32, d).times(o[d], p);
        }
    }
    l = both_halves_sum(l);
    const int64_t row = (int64_t)R.q * A.heads + R.head;
    const int64_t at = (int64_t)split * A.nq * A.heads + row;

    if (WM == 1) {
        // the four wavefronts' parts of the same rows, scaled to a common maximum
        if (h == 0) {
            jm[w][lane & 31] = m;
            jl[w][lane & 31] = l;
        }
        __syncthreads();
        float mt = -INFINITY, lt = 0.f;
#pragma unroll
        for (int u = 0; u < 4; u++) mt = fmaxf(mt, jm[u][lane & 31]);
        const float mb = mt == -INFINITY ? 0.f : mt;
#pragma unroll
        for (int u = 0; u < 4; u++) lt += jl[u][lane & 31] * exp2_fast(jm[u][lane & 31] - mb);
        const float f = exp2_fast(m - mb);
#pragma unroll
        for (int d = 0; d < DP / 32; d++)
#pragma unroll
            for (int i = 0; i < 16; i++) o[d][i] *= f;
        float r[DP / 32][4];
        sum_waves<DP>(reinterpret_cast<float *>(lds), o, w, r);
        if (!R.live) return;
        const float f2 = A.splits > 1 ? 1.f : inverse(lt);
#pragma unroll
        for (int d = 0; d < DP / 32; d++) {
            const int col = 32 * d + 8 * w + 4 * h;
#pragma unroll
            for (int e = 0; e < 4; e++) r[d][e] *= f2;
            if (A.splits > 1) Mma<float>::store4(A.part + at * DP + col, r[d]);
            else store_out<T>(A, row, col, r[d]);
        }
        m = mt;
        l = lt;
        if (w != 0) return;
    } else {
        if (!R.live || !busy) return;
        const float f2 = inverse(l);      // (128 rows a workgroup are never split)
#pragma unroll
        for (int d = 0; d < DP / 32; d++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const int col = 32 * d + 8 * g + 4 * h;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; e++) v[e] = o[d][4 * g + e] * f2;
                store_out<T>(A, row, col, v);
            }
    }
    if (h != 0) return;
    if (WM == 1 && A.splits > 1) {
        A.part_ml[2 * at] = m;
        A.part_ml[2 * at + 1] = l;
    } else if (A.lse) {
        A.lse[row] = log_sum(m, l);
    }
}

// Joins the splits of a row: a workgroup per (row, head), a lane per element, the
// wavefronts take the splits in turn (there are splits only where rows are few).  A
// launch's latency bounds it: 5 us for lifelong's 32 rows of 64 splits.
template <typename T, int DP>
__global__ __launch_bounds__(kAttnThreads) void attn_join(AttnArgs A)
{
    constexpr int G = kAttnThreads / DP;      // splits side by side
    __shared__ float sm[kSplitsMax], sl[kSplitsMax], so[G][DP];
    const int64_t row = blockIdx.x, n = (int64_t)A.nq * A.heads;
    const int t = threadIdx.x, d = t % DP, g = t / DP;
    for (int u = t; u < A.splits; u += kAttnThreads) {
        sm[u] = A.part_ml[2 * (u * n + row)];
        sl[u] = A.part_ml[2 * (u * n + row) + 1];
    }
    __syncthreads();
    float m = -INFINITY;
    for (int u = 0; u < A.splits; u++) m = fmaxf(m, sm[u]);
    const float mb = m == -INFINITY ? 0.f : m;
    float o = 0.f;
#pragma unroll 8
    for (int u = g; u < A.splits; u += G) o += A.part[(u * n + row) * DP + d] * exp2_fast(sm[u] - mb);
    so[g][d] = o;
    __syncthreads();
    if (g != 0) return;
    float l = 0.f;
    for (int u = 0; u < A.splits; u++) l += sl[u] * exp2_fast(sm[u] - mb);
    o = 0.f;
#pragma unroll
    for (int u = 0; u < G; u++) o += so[u][d];
    o *= inverse(l);
    if (d < A.dim) {
        Mma<T>::store1(static_cast<T *>(A.out) + row * A.dim + d, o);
        if (sizeof(T) == 2 && A.rest)
            Mma<T>::store1(static_cast<T *>(A.rest) + row * A.dim + d, o - bf16_lo(bf16_rne(o)));
    }
    if (d == 0 && A.lse) A.lse[row] = log_sum(m, l);
}

// ------------------------------------------------------- backward: queries

// dq_i = scale sum_j p_ij (dP_ij - D_i) k_j with D_i = o_i.dO_i, and along with it
// delta_i = D_i + sum_j p_ij (dP_ij - D_i), which the gradients of keys and bias use.
// D is delta up to the rounding of the probabilities that made the output (the output's
// own rounding is put back, from `rest`).  dq needs no more; but the bias gradient is
// a sum of score gradients over many rows, each row's adding up to zero, and would drown
// in that rounding: taken again from the probabilities in fp32, delta costs one addition
// a pair.  (Correcting dq for it too, by sum_j p_ij k_j, would be a fourth product.)
// dS enters its product in T, as q and k do.
// The walk is the forward's, and so is what bounds it.  Two sequences 258 us, 580 TFLOP/s
// of its three products (without a bias 198); ranking 52 us (43).
template <typename T, int DP, int WM>
__global__ __launch_bounds__(kAttnThreads, (KeyWalk<T, DP, WM>::kWaves)) void attn_backward_q(AttnArgs A)
{
    using KW = KeyWalk<T, DP, WM>;
    using TL = Tile<T, DP>;
    constexpr int SUBS = KW::KT / 32;
    __shared__ __align__(1024) u32x4_t lds[KW::kLds > 1024 ? KW::kLds : 1024];
    __shared__ int lbnd[kBucketsMax];
    __shared__ __align__(16) int kpos[4][32 * SUBS];
    __shared__ float jd[4][32];
    extern __shared__ float lb[];

    const Task job = task(A);
    const int split = job.split, kvh = job.kvh;
    if (kvh >= A.kv_heads) return;
    Bias B;
    B.take(A, kvh);
    const SegTile s = seg_find<WM * 32>(A.qo, A.nq, A.ko, A.nk, A.samples, A.group, job.tile);
    if (s.row0 >= s.rows) return;
    const int lane = lane_id(), h = lane >> 5, w = uniform((int)(threadIdx.x >> 6));
    const int r0 = s.row0 + (WM == 4 ? w * 32 : 0);
    const bool busy = r0 < s.rows;

    Row R = query_row(A, s, kvh, r0);
    const int64_t row = (int64_t)R.q * A.heads + R.head;
    Frag<T, DP> qf, df;
    load_frag<T, DP>(qf, static_cast<const T *>(A.q) + (int64_t)R.q * A.qs + R.head * A.qh, A.dim, A.vec, R.live);
    load_frag<T, DP>(df, static_cast<const T *>(A.dout) + (int64_t)R.q * A.ds + R.head * A.dh, A.dim, A.vec, R.live);
    float lse = R.live ? *gp(A.lse + row) : INFINITY, D = 0.f;
    KW walk(A, lds, kvh, w, s.o0, s.o1, split);
    walk.start();
    B.put(A, kvh, lb, lbnd);
    R.range();
    // a row without keys has no gradient, whatever arrives for its output
    if (lse == -INFINITY)
#pragma unroll
        for (int c = 0; c < TL::CH / 2; c++) df[c] = u32x4_t{0, 0, 0, 0};
    {
        Frag<T, DP> of;
        load_frag<T, DP>(of, static_cast<const T *>(A.out) + row * A.dim, A.dim, A.ovec, R.live);
#pragma unroll
        for (int c = 0; c < TL::CH / 2; c++) D += Mma<T>::dot(of[c], df[c]);
        if (sizeof(T) == 2) {
            load_frag<T, DP>(of, static_cast<const T *>(A.rest) + row * A.dim, A.dim, A.ovec, R.live);
#pragma unroll
            for (int c = 0; c < TL::CH / 2; c++) D += Mma<T>::dot(of[c], df[c]);
        }
        D = both_halves_sum(D);
    }
    // a row without keys has lse = -inf: exp2(score - inf) keeps its weights zero
    lse = lse == -INFINITY ? INFINITY : lse * kLog2e;
    if (A.bias) __syncthreads();      // the bias table
    BucketRun run{0, INT32_MAX, INT32_MIN};
    float b_run = 0.f;
    if (A.bias && walk.at < walk.end) {
        // the first keys' bucket, while they are on their way
        run.set(B, lbnd, B.bucket(sub_sat(R.r.lo, half_range(walk.pos_next).hi)));
        b_run = lb[run.m * A.group + R.g] * A.c;
    }

    float e = 0.f;                         // sum p (dP - D)
    f32x16_t x[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; d++) x[d] = f32x16_t{};

    for (; walk.at < walk.end; walk.leave()) {
        // no branch around the products, also where a wavefront has no rows (their weights
        // are zeros): accumulators that live across one are moved between the halves of the
        // register file at every step
        walk.enter();
        const u32x4_t *lk = walk.k_tile(), *lv = walk.v_tile();
        uint64_t in_run = A.bias ? run.covers(sub_sat(R.r.lo, walk.pos), sub_sat(R.r.hi, walk.pos)) : ~0ull;
        if (~in_run) {
            kpos[w][lane & (32 * SUBS - 1)] = walk.pos;
            wave_sync();
        }
#pragma unroll DP * sizeof(T) > 128 ? 1 : SUBS
        for (int u = 0; u < SUBS; u++) {
            const uint32_t keep = (uint32_t)(walk.keep >> (32 * u));
            f32x16_t sc = f32x16_t{}, dp;
#pragma unroll
            for (int i = 0; i < 16; i++) dp[i] = -D;
            float b = b_run;
            if (!kBiasFirst<T>) products<T, DP>(sc, lk, u * 32, qf);
            if (~in_run >> (32 * u) & 0xFFFFFFFFu) {
                mixed_bias<T>(A, B, lb, lbnd, R, kpos[w], walk.pos, u, true, run, sc, b, b_run);
                if (u + 1 < SUBS) in_run = run.covers(sub_sat(R.r.lo, walk.pos), sub_sat(R.r.hi, walk.pos));
            }
            if (kBiasFirst<T>) products<T, DP>(sc, lk, u * 32, qf);
            products<T, DP>(dp, lv, u * 32, df);
            b -= lse;
#pragma unroll
            for (int i = 0; i < 16; i++) sc[i] = exp2_fast(fmaf(sc[i], A.c, b));
            if (keep != 0xFFFFFFFFu) {
                const uint32_t mine = keep >> (4 * h);
#pragma unroll
                for (int i = 0; i < 16; i++) sc[i] = mine >> (8 * (i >> 2) + (i & 3)) & 1 ? sc[i] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 16; i++) {
                dp[i] *= sc[i];
                e += dp[i];
            }
            const typename Mma<T>::Pack ds = Mma<T>::pack(dp);
#pragma unroll
            for (int d = 0; d < DP / 32; d++) typename Mma<T>::template Rows<DP>(lk, u * 32, d).times(x[d], ds);
        }
    }
    e = both_halves_sum(e);
    const int64_t at = (int64_t)split * A.nq * A.heads + row;
    T *dq = static_cast<T *>(A.dq) + row * A.dim;
    if (WM == 1) {
        if (h == 0) jd[w][lane & 31] = e;
        float r[DP / 32][4];
        sum_waves<DP>(reinterpret_cast<float *>(lds), x, w, r);
        e = (jd[0][lane & 31] + jd[1][lane & 31]) + (jd[2][lane & 31] + jd[3][lane & 31]);
        if (!R.live) return;
#pragma unroll
        for (int d = 0; d < DP / 32; d++) {
            const int col = 32 * d + 8 * w + 4 * h;
#pragma unroll
            for (int i = 0; i < 4; i++) r[d][i] *= A.scale;
            if (A.splits > 1) Mma<float>::store4(A.part + at * DP + col, r[d]);
            else store_part(dq, col, A.dim, r[d]);
        }
        if (w != 0) return;
    } else {
        if (!R.live || !busy) return;
#pragma unroll
        for (int d = 0; d < DP / 32; d++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const int col = 32 * d + 8 * g + 4 * h;
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; i++) v[i] = A.scale * x[d][4 * g + i];
                store_part(dq, col, A.dim, v);
            }
    }
    if (h != 0) return;
    if (WM == 1 && A.splits > 1) {
        A.part_ml[2 * at] = D;
        A.part_ml[2 * at + 1] = e;
    } else {
        A.delta[row] = D + e;
    }
}

// dq and delta of a row from its splits, a workgroup per (row, head) as in attn_join
template <typename T, int DP>
__global__ __launch_bounds__(kAttnThreads) void attn_join_q(AttnArgs A)
{
    constexpr int G = kAttnThreads / DP;
    __shared__ float so[G][DP];
    const int64_t row = blockIdx.x, n = (int64_t)A.nq * A.heads;
    const int t = threadIdx.x, d = t % DP, g = t / DP;
    float x = 0.f, e = 0.f;
#pragma unroll 8
    for (int u = g; u < A.splits; u += G) x += A.part[(u * n + row) * DP + d];
    so[g][d] = x;
    __syncthreads();
    if (g != 0) return;
    x = 0.f;
#pragma unroll
    for (int u = 0; u < G; u++) x += so[u][d];
    for (int u = 0; u < A.splits; u++) e += A.part_ml[2 * (u * n + row) + 1];
    if (d < A.dim) Mma<T>::store1(static_cast<T *>(A.dq) + row * A.dim + d, x);
    if (d == 0) A.delta[row] = A.part_ml[2 * row] + e;
}

// ---------------------------------------------------------- backward: keys

// 32 rows, one per lane & 31 and DP elements long as the products leave them (times f),
// into memory rows `stride` elements apart: through a tile, so that neighbouring lanes
// write neighbouring 16 bytes.  Rows from `rows` on are left out; a row that is not `live` is
// zero.
template <typename T, int DP>
__device__ __forceinline__ void store_rows(T *base, int64_t stride, int dim, bool vec, int rows,
                                           const f32x16_t (&x)[DP / 32], float f, bool live, u32x4_t *tile)
{
    using TL = Tile<T, DP>;
    const int l = lane_id(), r = l & 31, h = l >> 5;
#pragma unroll
    for (int d = 0; d < DP / 32; d++)
#pragma unroll
        for (int g = 0; g < 4; g++) {
            const int col = 32 * d + 8 * g + 4 * h;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = f * x[d][4 * g + e];
            if (vec) lds_write(lds_address(tile) + 16 * TL::at(r, col / TL::E) + col % TL::E * (int)sizeof(T), Mma<T>::pack4(v));
            else if (r < rows) {
#pragma unroll
                for (int e = 0; e < 4; e++) v[e] = live ? v[e] : 0.f;
                store_part(base + r * stride, col, dim, v);
            }
        }
    if (!vec) return;
    const uint32_t alive = (uint32_t)__ballot(live);
    wave_sync();
    constexpr int PER = 64 / TL::CH;                    // rows per store
#pragma unroll
    for (int j = 0; j < 32 / PER; j++) {
        const int row = j * PER + l / TL::CH, c = (l % TL::CH) ^ swizzle<TL::CH>(row);
        u32x4_t v = tile[j * 64 + l];
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = alive >> row & 1 ? v[e] : 0;
        if (row < rows && c * TL::E < dim) *gp(reinterpret_cast<u32x4_t *>(base + row * stride) + c) = v;
    }
    wave_sync();
}

// distances of 16 query rows (in the order of a block) from the lane's key
__device__ __forceinline__ void distances(const int *qpos, int kpos, int (&x)[16])
{
    const int h = lane_id() >> 5;
#pragma unroll
    for (int g = 0; g < 4; g++) {
        const int4 q = *reinterpret_cast<const int4 *>(qpos + 8 * g + 4 * h);
        x[4 * g] = sub_sat(q.x, kpos);
        x[4 * g + 1] = sub_sat(q.y, kpos);
        x[4 * g + 2] = sub_sat(q.z, kpos);
        x[4 * g + 3] = sub_sat(q.w, kpos);
    }
}

// A workgroup owns 128 keys of one key head, 32 a wavefront (one per lane & 31), K
// and V in registers, and walks all query rows of the sample, one head of the group
// after the other, 32 rows a stage: dk and dv need no sum across workgroups.  Rows
// arrive in LDS a stage ahead, as the keys do in the other kernels.
// Rows of 256 bytes leave V in LDS: with V in registers too they would need more than
// 256, and past those the accumulators move back and forth (see KeyWalk::kWaves; two
// sequences 582 us with V in registers, 506 with it in LDS, when this was chosen).
// Two sequences 470 to 505 us by their positions, 395 to 425 TFLOP/s of its four products
// (without a bias 284): products, weights and the bias gradient's sums take turns in two
// wavefronts a SIMD.  A block in one bucket adds its 16 score gradients to a sum in a
// register; the sum goes to LDS when the bucket changes (LDS additions per pair instead:
// 1237 -> 2537 us).  Ranking 92 us (59), 1.6 TB/s of the keys' 146 MB: with 2 or 3 stages
// a workgroup the time goes to the latency of its first loads and to blocks that span
// several buckets.  Clearing rows without keys costs 1.5 of the 92 us, zeros for masked keys
// 1.
template <typename T, int DP>
__global__ __launch_bounds__(kAttnThreads, (DP * sizeof(T) <= 256 ? 2 : 1)) void attn_backward_k(AttnArgs A)
{
    using TL = Tile<T, DP>;
    constexpr bool kSpill = DP * sizeof(T) == 256;
    __shared__ __align__(1024) u32x4_t lvk[kSpill ? 128 * TL::CH : 1];
    constexpr int kWords = 32 * TL::CH;
    __shared__ __align__(1024) u32x4_t lds[2][2][kWords];             // [stage & 1][q, dout]
    __shared__ __align__(16) float nlse[2][32], ndelta[2][32];      // - lse in log2 (or -inf), - delta
    __shared__ __align__(16) int qpos[2][32];
    __shared__ int qlo[2], qhi[2];
    __shared__ int lbnd[kBucketsMax];
    __shared__ float acc[4][kBucketsMax];
    extern __shared__ float lb[];

    const Task job = task(A);
    const int kvh = job.kvh;
    const int tile = job.tile;
    if (kvh >= A.kv_heads) return;
    Bias B;
    B.take(A, kvh);
    const SegTile s = seg_find<128>(A.ko, A.nk, A.qo, A.nq, A.samples, 1, tile);
    const bool idle = s.row0 >= s.rows;
    if (idle && !A.dbias_part) return;
    const int lane = lane_id(), h = lane >> 5, w = uniform((int)(threadIdx.x >> 6));
    const int q0 = s.o0, q1 = idle ? s.o0 : s.o1;
    const int64_t stages = (int64_t)((q1 - q0 + 31) / 32) * A.group;

    // a stage: head g of the group, 32 rows from `row`
    struct Stage {
        int g, row;
        int64_t i;
    };
    auto after = [&](Stage z) {
        z.i++;
        z.row += 32;
        if (z.row >= q1) {
            z.row = q0;
            z.g++;
        }
        return z;
    };
    // a row without keys (lse = -inf) becomes zeros once it has arrived: its weights of zero
    // must not meet an infinity or NaN
    float b_lse = 0.f;
    auto bring = [&](const Stage &z, int to) {
        if (z.i >= stages) return;
        // wavefronts 0 and 1 bring the halves of q, 2 and 3 those of dout
        const int head = kvh * A.group + z.g, half = (w & 1) * 16;
        const int row = z.row + half, left = q1 - row;
        const uint64_t keep = left <= 0 ? 0 : left >= 16 ? 0xFFFF : (1u << left) - 1;
        const T *p = w < 2 ? static_cast<const T *>(A.q) + head * A.qh + (int64_t)row * A.qs
                           : static_cast<const T *>(A.dout) + head * A.dh + (int64_t)row * A.ds;
        bring_rows<T, DP, 16>(p, w < 2 ? A.qs : A.ds, A.dim, A.vec, keep, lds[to][w >> 1], half);
        b_lse = *gp(A.lse + (int64_t)min(row + (lane & 15), q1 - 1) * A.heads + head);
    };
    float n_lse = 0.f, n_delta = 0.f;
    int n_pos = 0;
    bool n_in = false;
    auto look = [&](const Stage &z) {       // wavefront 0: what goes with the rows
        if (z.i >= stages) return;
        const int row = z.row + (lane & 31);
        n_in = row < q1;
        const int64_t at = (int64_t)(n_in ? row : q1 - 1) * A.heads + kvh * A.group + z.g;
        n_lse = *gp(A.lse + at);
        n_delta = *gp(A.delta + at);
        if (A.bias) n_pos = *gp(A.qp + (n_in ? row : q1 - 1));
    };
    auto tell = [&](int to) {
        // a row without keys, and one past the end: weights of zero
        nlse[to][lane & 31] = n_in && n_lse != -INFINITY ? -n_lse * kLog2e : -INFINITY;
        ndelta[to][lane & 31] = n_in ? -n_delta : 0.f;
        if (!A.bias) return;
        qpos[to][lane & 31] = n_pos;
        const Range r = half_range(n_pos);
        qlo[to] = r.lo;
        qhi[to] = r.hi;
    };

    Stage now{0, q0, 0}, next = after(now), then = after(next);
    bring(now, 0);
    if (w == 0) look(now);
    if (A.dbias_part)
        for (int i = threadIdx.x; i < 4 * kBucketsMax; i += kAttnThreads) (&acc[0][0])[i] = 0.f;
    const int r = s.row0 + 32 * w + (lane & 31);
    const bool in = r < s.rows;
    const int64_t key = s.base + (in ? r : s.rows - 1);
    const int kpos = A.bias && !idle ? *gp(A.kp + key) : 0;
    const int qpos0 = A.bias && stages ? *gp(A.qp + q0) : 0;
    const bool live = in && !idle && (!A.mask || *gp(A.mask + key));
    Frag<T, DP> kf, vf;
    load_frag<T, DP>(kf, static_cast<const T *>(A.k) + (live ? key * A.ks + kvh * A.kh : 0), A.dim, A.vec, live);
    load_frag<T, DP>(vf, static_cast<const T *>(A.v) + (live ? key * A.vs + kvh * A.vh : 0), A.dim, A.vec, live);
    if (kSpill) {
#pragma unroll
        for (int c = 0; c < TL::CH / 2; c++) lvk[TL::at(32 * w + (lane & 31), 2 * c + h)] = vf[c];
        wave_sync();
    }
    B.put(A, kvh, lb, lbnd);
    Range kr{0, 0};
    if (A.bias) kr = half_range(kpos);
    if (w == 0) {
        tell(0);
        look(next);
    }
    if (A.bias) __syncthreads();      // the bias table

    f32x16_t dk[DP / 32], dv[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; d++) dk[d] = dv[d] = f32x16_t{};
    // score gradients of the bucket at hand, a sum per lane until the bucket changes
    BucketRun run{0, INT32_MAX, INT32_MIN};
    float b_run = live ? 0.f : -INFINITY, sum_run = 0.f;
    if (A.bias && stages) {
        run.set(B, lbnd, B.bucket(sub_sat(qpos0, kr.hi)));
        b_run = live ? lb[run.m * A.group] : -INFINITY;
    }
    // (an LDS addition without an answer; only this wavefront adds to its own row, in order)
    auto settle = [&](int m, float sum) {
        sum = wave_sum(live ? sum : 0.f);
        if (lane == 0) __hip_atomic_fetch_add(&acc[w][m], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    };

    for (; now.i < stages; now = next, next = then, then = after(then)) {
        const int cur = (int)(now.i & 1);
        arrived();
        if (const uint32_t dead = (uint32_t)__ballot(b_lse == -INFINITY) & 0xFFFF)
            for (int i = lane; i < 16 * TL::CH; i += 64)
                if (dead >> (i / TL::CH) & 1) lds[cur][w >> 1][(w & 1) * 16 * TL::CH + i] = u32x4_t{0, 0, 0, 0};
        __syncthreads();
        bring(next, cur ^ 1);
        if (w == 0) {
            tell(cur ^ 1);
            look(then);
        }
        const u32x4_t *lq = lds[cur][0], *ld = lds[cur][1];
        {
            f32x16_t start, dp = block_order(ndelta[cur]);
#pragma unroll
            for (int i = 0; i < 16; i++) start[i] = b_run;
            int lo = run.m, hi = run.m;
            if (A.bias && ~run.covers(sub_sat(qlo[cur], kpos), sub_sat(qhi[cur], kpos)) != 0) {
                // as mixed_bias, with one key and 16 rows a lane
                lo = B.bucket(sub_sat(qlo[cur], kr.hi));
                hi = B.bucket(sub_sat(qhi[cur], kr.lo));
                if (A.dbias_part && lo != run.m) {
                    settle(run.m, sum_run);
                    sum_run = 0.f;
                }
                run.set(B, lbnd, hi);
                float v = lb[lo * A.group + now.g];
                v = live ? v : -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; i++) start[i] = v;
                if (lo != hi) {
                    int x[16];
                    distances(qpos[cur], kpos, x);
                    for (int m = lo; m < hi; m++) {
                        const int edge = lbnd[m];
                        v = live ? lb[(m + 1) * A.group + now.g] : -INFINITY;
#pragma unroll
                        for (int i = 0; i < 16; i++) start[i] = x[i] >= edge ? v : start[i];
                    }
                }
                b_run = v;
            }
            f32x16_t sc = kBiasFirst<T> ? start : f32x16_t{};
            products<T, DP>(sc, lq, 0, kf);
            if (!kBiasFirst<T>) sc += start;
            const f32x16_t nl = block_order(nlse[cur]);
            if (kSpill) products<T, DP>(dp, ld, 0, lvk, 32 * w);
            else products<T, DP>(dp, ld, 0, vf);
#pragma unroll
            for (int i = 0; i < 16; i++) {
                sc[i] = exp2_fast(fmaf(sc[i], A.c, nl[i]));
                dp[i] *= sc[i];
            }
            const typename Mma<T>::Pack p = Mma<T>::pack(sc), ds = Mma<T>::pack(dp);
#pragma unroll
            for (int d = 0; d < DP / 32; d++) {
                typename Mma<T>::template Rows<DP>(ld, 0, d).times(dv[d], p);
                typename Mma<T>::template Rows<DP>(lq, 0, d).times(dk[d], ds);
            }
            if (A.dbias_part) {
                if (lo != hi) {
                    // each bucket's own terms: what a boundary leaves below it is taken out.  (What
                    // lies below one less what lay below the one before costs three operations a
                    // pair, not four, two sequences 461 us for 483; but a small sum beside a large
                    // one would lose its digits.)
                    int x[16];
                    distances(qpos[cur], kpos, x);
                    for (int m = lo; m < hi; m++) {
                        const int edge = lbnd[m];
                        float sum = 0.f;
#pragma unroll
                        for (int i = 0; i < 16; i++) {
                            const bool below = x[i] < edge;
                            sum += below ? dp[i] : 0.f;
                            dp[i] = below ? 0.f : dp[i];
                        }
                        settle(m, sum_run + sum);
                        sum_run = 0.f;
                    }
                }
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 16; i++) sum += dp[i];
                sum_run += sum;
            }
        }
        const int last_m = run.m;
        if (next.g != now.g) run = BucketRun{last_m, INT32_MAX, INT32_MIN};     // another head, another bias
        if (A.dbias_part && next.g != now.g) {       // a head of the group is done
            settle(last_m, sum_run);
            sum_run = 0.f;
            __syncthreads();
            float *to = A.dbias_part + ((int64_t)tile * A.heads + kvh * A.group + now.g) * A.buckets;
            for (int m = threadIdx.x; m < A.buckets; m += kAttnThreads) {
                to[m] = (acc[0][m] + acc[1][m]) + (acc[2][m] + acc[3][m]);
                acc[0][m] = acc[1][m] = acc[2][m] = acc[3][m] = 0.f;
            }
            __syncthreads();
        }
    }
    if (A.dbias_part && stages == 0)
        for (int i = threadIdx.x; i < A.buckets * A.group; i += kAttnThreads)
            A.dbias_part[((int64_t)tile * A.heads + kvh * A.group) * A.buckets + i] = 0.f;
    if (idle || !A.dk) return;
    const int rows = s.rows - (s.row0 + 32 * w);
    const int64_t at = ((int64_t)(s.base + s.row0 + 32 * w) * A.kv_heads + kvh) * A.dim;
    u32x4_t *mine = lds[w >> 1][w & 1];
    __syncthreads();                  // the last stage's rows are read
    store_rows<T, DP>(static_cast<T *>(A.dk) + at, (int64_t)A.kv_heads * A.dim, A.dim, A.gvec, rows, dk, A.scale, live,
                      mine);
    store_rows<T, DP>(static_cast<T *>(A.dv) + at, (int64_t)A.kv_heads * A.dim, A.dim, A.gvec, rows, dv, 1.f, live, mine);
}

// dbias[m, head] = sum of the workgroups' parts, in a fixed order (no atomics: the result
// is the same every time): a workgroup per (head, 32 buckets), 32 tiles side by side.
// 4 to 5 us: a launch's latency and a few dependent loads; 12 us for 2500 tiles.
constexpr int kBiasJoin = 1024;
__global__ __launch_bounds__(kBiasJoin) void attn_join_bias(AttnArgs A, float *dbias)
{
    __shared__ float part[32][32];
    const int head = blockIdx.x, t = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int m = blockIdx.y * 32 + t, mc = m < A.buckets ? m : A.buckets - 1;
    float sum = 0.f;
#pragma unroll 8
    for (int u = g; u < A.tiles; u += 32) sum += *gp(A.dbias_part + ((int64_t)u * A.heads + head) * A.buckets + mc);
    part[g][t] = sum;
    __syncthreads();
    if (g != 0 || m >= A.buckets) return;
    sum = 0.f;
#pragma unroll
    for (int u = 0; u < 32; u++) sum += part[u][t];
    dbias[(int64_t)m * A.heads + head] = sum;
}

}  // namespace emb

using namespace emb;

namespace {

size_t pad256(size_t x) { return (x + 255) & ~size_t(255); }

// How the kernels that walk the keys are cut: 32 or 128 query rows a workgroup (WM = 1
// or 4), and the number of workgroups that share the keys of one set of rows.
// 128 rows read K and V from L2 a quarter as often, but leave rows unused in samples of
// few and fill the chip only with enough sets of rows.  Forward in us, 32 / 128 rows:
// two sequences 449 / 201 (944 sets of 128), many candidates 61 / 59 (364 sets), serving
// 121 / 166, ranking 45 / 60; fp32 training of 16 samples of 1..64 queries 62 / 109 in
// all three kernels.
// Splits pay while the sets alone leave the chip's 512 places (two workgroups a CU) empty,
// and cost partial results and a launch: lifelong with 1, 8, 32, 64 splits takes 1297,
// 182, 88, 89 us, where many candidates with 2 take 99 us for 61, and ranking 236 for 193.
// A split of under 256 keys would be two steps long.
struct AttnPlan {
    int wm, splits;
    int64_t tiles, key_tiles;
};

AttnPlan attn_plan(const emb_attention *a)
{
    AttnPlan p{};
    const int group = a->heads / a->kv_heads;
    const int64_t rows = a->n_q * group, samples = a->samples > 0 ? a->samples : 1;
    const int64_t keys = a->n_k / samples;             // of the average sample
    const int64_t busy = std::min<int64_t>(samples, a->n_q);
    auto sets = [&](int per) { return std::max(rows / per + busy / 2, busy) * a->kv_heads; };
    p.wm = sets(128) >= 384 && rows / samples > 64 ? 4 : 1;
    p.tiles = seg_tiles(a->n_q, a->samples, group, 32 * p.wm);
    // (the sets that 128 rows take already leave no place for a second split)
    int64_t s = p.wm == 1 && sets(32) > 0 ? 512 / sets(32) : 1;
    s = std::min<int64_t>(s, keys / 256);
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(s, kSplitsMax));
    p.key_tiles = seg_tiles(a->n_k, a->samples, 1, 128);
    return p;
}

int padded_dim(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : 128; }

size_t forward_workspace(const emb_attention *a, const AttnPlan &p)
{
    if (p.splits == 1) return 0;
    const size_t rows = (size_t)p.splits * a->n_q * a->heads;
    return pad256(rows * padded_dim(a->dim) * 4) + pad256(rows * 8);
}

size_t backward_workspace(const emb_attention *a, const AttnPlan &p)
{
    size_t n = pad256((size_t)a->n_q * a->heads * 4);
    if (p.splits > 1) {
        const size_t rows = (size_t)p.splits * a->n_q * a->heads;
        n += pad256(rows * padded_dim(a->dim) * 4) + pad256(rows * 8);
    }
    if (a->buckets) n += pad256((size_t)p.key_tiles * a->heads * a->buckets * 4);
    return n;
}

emb_status attn_check(const emb_attention *a)
{
    if (!a) return fail(EMB_ERR_INVALID_ARG, "attention descriptor is NULL");
    if (a->dtype != EMB_F32 && a->dtype != EMB_BF16) return fail(EMB_ERR_INVALID_ARG, "attention: unknown dtype");
    if (a->heads <= 0 || a->kv_heads <= 0 || a->heads % a->kv_heads)
        return fail(EMB_ERR_INVALID_ARG, "attention: heads must be a positive multiple of kv_heads");
    if (a->dim <= 0) return fail(EMB_ERR_INVALID_ARG, "attention: dim must be >= 1");
    if (a->dim > 128) return fail(EMB_ERR_UNSUPPORTED, "attention: dim must be <= 128");
    if (a->samples < 0 || a->n_q < 0 || a->n_k < 0)
        return fail(EMB_ERR_INVALID_ARG, "attention: samples, n_q and n_k must be >= 0");
    if (a->n_q > kRowsMost / (a->heads / a->kv_heads) || a->n_k > kRowsMost || a->samples > (1 << 30))
        return fail(EMB_ERR_UNSUPPORTED,
                    "attention: n_q heads / kv_heads and n_k must be <= 2^31 - 65536, samples <= 2^30");
    if (a->heads > 65535) return fail(EMB_ERR_UNSUPPORTED, "attention: heads must be <= 65535");
    if (!(a->scale >= 1e-18f && a->scale <= 1e18f))
        return fail(EMB_ERR_INVALID_ARG, "attention: scale must be in [1e-18, 1e18]");
    if (a->buckets < 0) return fail(EMB_ERR_INVALID_ARG, "attention: buckets must be >= 0");
    if (a->buckets > kBucketsMax) return fail(EMB_ERR_UNSUPPORTED, "attention: buckets must be <= 256");
    if ((int64_t)a->buckets * (a->heads / a->kv_heads) > kBiasWords)
        return fail(EMB_ERR_UNSUPPORTED, "attention: buckets times heads per key head must be <= 4096");
    if (a->q_stride < 0 || a->q_head_stride < 0 || a->k_stride < 0 || a->k_head_stride < 0 || a->v_stride < 0 ||
        a->v_head_stride < 0)
        return fail(EMB_ERR_INVALID_ARG, "attention: strides must be >= 0");
    return EMB_OK;
}

emb_status attn_pointers(const emb_attention *a)
{
    const size_t el = a->dtype == EMB_BF16 ? 2 : 4;
    if (!a->q_offsets || !a->k_offsets || !aligned(a->q_offsets, 4) || !aligned(a->k_offsets, 4))
        return fail(EMB_ERR_INVALID_ARG, "attention: q_offsets and k_offsets must be given");
    if ((a->n_q && !a->q) || (a->n_k && (!a->k || !a->v)))
        return fail(EMB_ERR_INVALID_ARG, "attention: q, k and v must be given");
    if (!aligned(a->q, el) || !aligned(a->k, el) || !aligned(a->v, el))
        return fail(EMB_ERR_INVALID_ARG, "attention: q, k and v must be aligned to their elements");
    if (a->buckets) {
        if (!a->bias || (a->n_q && !a->q_pos) || (a->n_k && !a->k_pos) || (a->buckets > 1 && !a->boundaries))
            return fail(EMB_ERR_INVALID_ARG, "attention: a bias needs q_pos, k_pos and boundaries");
        if (!aligned(a->bias, 4) || !aligned(a->q_pos, 4) || !aligned(a->k_pos, 4) || !aligned(a->boundaries, 4))
            return fail(EMB_ERR_INVALID_ARG, "attention: bias, positions and boundaries must be 4-byte aligned");
    }
    return EMB_OK;
}

// rows that can be read in 16-byte pieces: whole pieces per row, every row aligned, and
// the 64 rows of a tile within the 2^31 bytes that one descriptor reaches
bool wide_rows(const void *p, int64_t stride, int64_t head_stride, int dim, size_t el)
{
    return stride < (int64_t(1) << 31) / 64 / (int64_t)el && aligned(p, 16) && stride * el % 16 == 0 && head_stride * el % 16 == 0 && dim * el % 16 == 0;
}

AttnArgs attn_args(const emb_attention *a, const AttnPlan &p)
{
    const size_t el = a->dtype == EMB_BF16 ? 2 : 4;
    AttnArgs A{};
    A.q = a->q;
    A.k = a->k;
    A.v = a->v;
    A.qs = a->q_stride;
    A.qh = a->q_head_stride;
    A.ks = a->k_stride;
    A.kh = a->k_head_stride;
    A.vs = a->v_stride;
    A.vh = a->v_head_stride;
    A.qo = a->q_offsets;
    A.ko = a->k_offsets;
    A.mask = a->mask;
    A.qp = a->q_pos;
    A.kp = a->k_pos;
    A.bnd = a->boundaries;
    A.bias = a->buckets ? a->bias : nullptr;
    A.nq = (int32_t)a->n_q;
    A.nk = (int32_t)a->n_k;
    A.samples = a->samples;
    A.heads = a->heads;
    A.kv_heads = a->kv_heads;
    A.group = a->heads / a->kv_heads;
    A.dim = a->dim;
    A.buckets = a->buckets;
    A.scale = a->scale;
    A.rscale = 1.f / a->scale;
    A.c = a->scale * kLog2e;
    A.vec = wide_rows(a->q, a->q_stride, a->q_head_stride, a->dim, el) &&
            wide_rows(a->k, a->k_stride, a->k_head_stride, a->dim, el) &&
            wide_rows(a->v, a->v_stride, a->v_head_stride, a->dim, el);
    A.splits = p.splits;
    A.tiles = (int32_t)p.tiles;
    // Neighbours in the order of work share keys (tiles of a sample) and so an XCD's L2:
    // each XCD takes one run of them (ranking 193 us, against 205 in runs of 16).  Splits
    // share nothing, and there few samples of unequal length even out in runs of 16
    // (lifelong 98 us, against 131).
    A.chunk = p.splits > 1 ? 16 : 0;
    return A;
}

emb_status launched(const char *what)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(EMB_ERR_HIP, std::string(what) + " launch: " + hipGetErrorString(e));
    return EMB_OK;
}

template <typename T, int DP>
emb_status forward_run(const AttnArgs &A, const AttnPlan &p, hipStream_t st)
{
    const size_t lds = (size_t)A.buckets * A.group * 4;
    const dim3 grid((unsigned)xcd_grid(p.tiles * A.kv_heads * p.splits, A.chunk)), block(kAttnThreads);
    if (p.wm == 4) hipLaunchKernelGGL((attn_forward<T, DP, 4>), grid, block, lds, st, A);
    else hipLaunchKernelGGL((attn_forward<T, DP, 1>), grid, block, lds, st, A);
    if (p.splits > 1)
        hipLaunchKernelGGL((attn_join<T, DP>), dim3((unsigned)((int64_t)A.nq * A.heads)), block, 0, st, A);
    return launched("attention forward");
}

template <typename T, int DP>
emb_status backward_run(const AttnArgs &A0, const AttnPlan &p, float *dbias, hipStream_t st)
{
    AttnArgs A = A0;
    const size_t lds = (size_t)A.buckets * A.group * 4;
    const dim3 block(kAttnThreads);
    if (A.nq) {
        const dim3 grid((unsigned)xcd_grid(p.tiles * A.kv_heads * p.splits, A.chunk));
        if (p.wm == 4) hipLaunchKernelGGL((attn_backward_q<T, DP, 4>), grid, block, lds, st, A);
        else hipLaunchKernelGGL((attn_backward_q<T, DP, 1>), grid, block, lds, st, A);
        if (p.splits > 1)
            hipLaunchKernelGGL((attn_join_q<T, DP>), dim3((unsigned)((int64_t)A.nq * A.heads)), block, 0, st, A);
    }
    A.tiles = (int32_t)p.key_tiles;
    A.splits = 1;
    if (A.dk || dbias)
        hipLaunchKernelGGL((attn_backward_k<T, DP>), dim3((unsigned)xcd_grid(p.key_tiles * A.kv_heads, A.chunk)), block, lds, st, A);
    if (dbias)
        hipLaunchKernelGGL(attn_join_bias, dim3((unsigned)A.heads, (unsigned)((A.buckets + 31) / 32)),
                           dim3(kBiasJoin), 0, st, A,
                           dbias);
    return launched("attention backward");
}

// a launch's threads are counted in 32 bits (and the grids are rounded up to a multiple
// of the XCDs and chunks)
bool grid_fits(const emb_attention *a, const AttnPlan &p)
{
    const double most = 4294967295.0 / kAttnThreads - 1024;
    return (double)p.tiles * a->kv_heads * p.splits <= most && (double)p.key_tiles * a->kv_heads <= most &&
           (double)a->n_q * a->heads <= (p.splits > 1 ? most : 2147483647.0);
}

}  // namespace

extern "C" emb_status emb_attention_query(const emb_attention *a, size_t *forward_bytes, size_t *backward_bytes)
{
    const emb_status s = attn_check(a);
    if (s != EMB_OK) return s;
    if (!forward_bytes || !backward_bytes)
        return fail(EMB_ERR_INVALID_ARG, "attention: output pointers must be given");
    const AttnPlan p = attn_plan(a);
    *forward_bytes = forward_workspace(a, p);
    *backward_bytes = backward_workspace(a, p);
    return EMB_OK;
}

extern "C" emb_status emb_attention_forward(const emb_attention *a, void *out, void *rest, float *lse,
                                            void *workspace, size_t workspace_bytes, void *stream)
{
    emb_status s = attn_check(a);
    if (s == EMB_OK) s = attn_pointers(a);
    if (s != EMB_OK) return s;
    if (a->n_q == 0) return EMB_OK;
    const size_t el = a->dtype == EMB_BF16 ? 2 : 4;
    const size_t al = a->dim % 4 == 0 ? 4 * el : el;
    if (!out || !aligned(out, al) || !aligned(rest, al) || !aligned(lse, 4))
        return fail(EMB_ERR_INVALID_ARG, "attention: out must be given, out and rest aligned to four elements");
    const AttnPlan p = attn_plan(a);
    if (!grid_fits(a, p)) return fail(EMB_ERR_UNSUPPORTED, "attention: more than 2^24 - 1024 workgroups of rows");
    const size_t need = forward_workspace(a, p);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return fail(EMB_ERR_WORKSPACE, "attention: the workspace is smaller than the query returned, or not 256-byte aligned");
    AttnArgs A = attn_args(a, p);
    A.out = out;
    A.rest = rest;
    A.lse = lse;
    if (need) {
        A.part = static_cast<float *>(workspace);
        A.part_ml = reinterpret_cast<float *>(
            static_cast<char *>(workspace) + pad256((size_t)p.splits * a->n_q * a->heads * padded_dim(a->dim) * 4));
    }
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int dp = padded_dim(a->dim);
    if (a->dtype == EMB_BF16)
        return dp == 32   ? forward_run<uint16_t, 32>(A, p, st)
               : dp == 64 ? forward_run<uint16_t, 64>(A, p, st)
                          : forward_run<uint16_t, 128>(A, p, st);
    return dp == 32   ? forward_run<float, 32>(A, p, st)
           : dp == 64 ? forward_run<float, 64>(A, p, st)
                      : forward_run<float, 128>(A, p, st);
}

extern "C" emb_status emb_attention_backward(const emb_attention *a, const void *out, const void *rest, const float *lse, const void *dout,
                                             int64_t dout_stride, int64_t dout_head_stride, void *dq, void *dk,
                                             void *dv, float *dbias, void *workspace, size_t workspace_bytes,
                                             void *stream)
{
    emb_status s = attn_check(a);
    if (s == EMB_OK) s = attn_pointers(a);
    if (s != EMB_OK) return s;
    const size_t el = a->dtype == EMB_BF16 ? 2 : 4;
    const size_t al = a->dim % 4 == 0 ? 4 * el : el;
    if (a->n_q && (!out || !lse || !dout || !dq))
        return fail(EMB_ERR_INVALID_ARG, "attention: out, lse, dout and dq must be given");
    if (a->n_q && a->dtype == EMB_BF16 && !rest)
        return fail(EMB_ERR_INVALID_ARG, "attention: the bf16 backward needs rest");
    if (!dk != !dv) return fail(EMB_ERR_INVALID_ARG, "attention: dk and dv are given together");
    if (dbias && !a->buckets) return fail(EMB_ERR_INVALID_ARG, "attention: dbias without a bias");
    if (!aligned(dout, el) || !aligned(out, el) || !aligned(rest, el) || !aligned(dq, al) || !aligned(dk, al) || !aligned(dv, al) || !aligned(lse, 4) ||
        !aligned(dbias, 4))
        return fail(EMB_ERR_INVALID_ARG, "attention: gradients must be aligned to four elements");
    if (dout_stride < 0 || dout_head_stride < 0) return fail(EMB_ERR_INVALID_ARG, "attention: strides must be >= 0");
    const AttnPlan p = attn_plan(a);
    if (!grid_fits(a, p)) return fail(EMB_ERR_UNSUPPORTED, "attention: more than 2^24 - 1024 workgroups of rows");
    const size_t need = backward_workspace(a, p);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return fail(EMB_ERR_WORKSPACE, "attention: the workspace is smaller than the query returned, or not 256-byte aligned");
    AttnArgs A = attn_args(a, p);
    A.dout = dout;
    A.ds = dout_stride;
    A.dh = dout_head_stride;
    A.vec = A.vec && wide_rows(dout, dout_stride, dout_head_stride, a->dim, el);
    A.out = const_cast<void *>(out);
    A.rest = const_cast<void *>(rest);
    A.ovec = wide_rows(out, a->dim, a->dim, a->dim, el) && wide_rows(rest, a->dim, a->dim, a->dim, el);
    A.gvec = wide_rows(dk, a->dim, a->dim, a->dim, el) && wide_rows(dv, a->dim, a->dim, a->dim, el);
    A.lse = const_cast<float *>(lse);
    A.dq = dq;
    A.dk = dk;
    A.dv = dv;
    char *ws = static_cast<char *>(workspace);
    A.delta = reinterpret_cast<float *>(ws);
    ws += pad256((size_t)a->n_q * a->heads * 4);
    if (p.splits > 1) {
        const size_t rows = (size_t)p.splits * a->n_q * a->heads;
        A.part = reinterpret_cast<float *>(ws);
        ws += pad256(rows * padded_dim(a->dim) * 4);
        A.part_ml = reinterpret_cast<float *>(ws);
        ws += pad256(rows * 8);
    }
    if (dbias) A.dbias_part = reinterpret_cast<float *>(ws);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int dp = padded_dim(a->dim);
    if (a->dtype == EMB_BF16)
        return dp == 32   ? backward_run<uint16_t, 32>(A, p, dbias, st)
               : dp == 64 ? backward_run<uint16_t, 64>(A, p, dbias, st)
                          : backward_run<uint16_t, 128>(A, p, dbias, st);
    return dp == 32   ? backward_run<float, 32>(A, p, dbias, st)
           : dp == 64 ? backward_run<float, 64>(A, p, dbias, st)
                      : backward_run<float, 128>(A, p, dbias, st);
}
