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
#include <algorithm>
#include <cmath>
#include <string>

#include "sequence.h"

namespace emb {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kBucketsMax = 256;
constexpr int kBiasWords = 4096;        // heads per key head x buckets held in LDS
constexpr int kAttnThreads = 256;

struct AttnArgs {
    const void *q, *k, *v, *dout;
    int64_t qs, qh, ks, kh, vs, vh, ds, dh;     // row and head strides in elements
    const int32_t *qo, *ko;                     // [samples + 1]
    const uint8_t *mask;                        // [n_k] or NULL
    const int32_t *qp, *kp, *bnd;               // positions, boundaries [buckets - 1]
    const float *bias;                          // [buckets, heads] or NULL
    int64_t nq, nk;
    int32_t samples, heads, kv_heads, group, dim, buckets;
    float scale, c;                             // c = scale * log2(e)
    int32_t vec;                                // rows can be read 16 bytes at a time
    int32_t splits;
    int64_t tiles;
    void *out;                                  // [n_q, heads, dim]
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
    // acc[d, lane] += sum over the block's 32 keys of tile[key, d] w[key, lane], for
    // d = 32 db ..: the tile's rows `r0 ..` are read transposed
    template <int DP>
    static __device__ __forceinline__ void transposed(f32x16_t &acc, const u32x4_t *tile, int r0, int db,
                                                      const Pack &w)
    {
        using TL = Tile<uint16_t, DP>;
        const int l = lane_id(), h = l >> 5;
#pragma unroll
        for (int kc = 0; kc < 2; kc++) {
            s16x8_t a;
#pragma unroll
            for (int jb = 0; jb < 2; jb++) {
                const int row = r0 + 16 * kc + 8 * jb + 4 * h + ((l & 15) >> 2);
                const int col = 32 * db + 16 * ((l >> 4) & 1) + 4 * (l & 3);
                const char *p = reinterpret_cast<const char *>(tile + TL::at(row, col >> 3)) + (col & 7) * 2;
                const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4_t *)(p));
#pragma unroll
                for (int e = 0; e < 4; e++) a[4 * jb + e] = v[e];
            }
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                          __builtin_bit_cast(bf16x8_t, w.w[kc]), acc, 0, 0, 0);
        }
    }
    static __device__ __forceinline__ void store4(uint16_t *p, const float *v)
    {
        *gp(reinterpret_cast<uint2 *>(p)) = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
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
    static __device__ __forceinline__ void transposed(f32x16_t &acc, const u32x4_t *tile, int r0, int db,
                                                      const Pack &w)
    {
        using TL = Tile<float, DP>;
        const int l = lane_id(), h = l >> 5, d = 32 * db + (l & 31);
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const int row = r0 + 8 * (i >> 2) + 4 * h + (i & 3);
            const float a = reinterpret_cast<const float *>(tile + TL::at(row, d >> 2))[d & 3];
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a, w.w[i], acc, 0, 0, 0);
        }
    }
    static __device__ __forceinline__ void store4(float *p, const float *v)
    {
        *gp(reinterpret_cast<float4 *>(p)) = make_float4(v[0], v[1], v[2], v[3]);
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
    const int l = lane_id(), h = l >> 5;
#pragma unroll
    for (int c = 0; c < TL::CH / 2; c++)
        Mma<T>::chunk(acc, tile[TL::at(r0 + (l & 31), 2 * c + h)], b[c]);
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

__device__ __forceinline__ float both_halves_max(float x) { return fmaxf(x, __shfl_xor(x, 32)); }
__device__ __forceinline__ float both_halves_sum(float x) { return x + __shfl_xor(x, 32); }
__device__ __forceinline__ float wave_sum(float x)
{
#pragma unroll
    for (int s = 32; s; s >>= 1) x += __shfl_xor(x, s);
    return x;
}
__device__ __forceinline__ int min32(int x)     // over the 32 lanes of a half
{
#pragma unroll
    for (int s = 16; s; s >>= 1) x = min(x, __shfl_xor(x, s));
    return x;
}
__device__ __forceinline__ int max32(int x)
{
#pragma unroll
    for (int s = 16; s; s >>= 1) x = max(x, __shfl_xor(x, s));
    return x;
}

// ------------------------------------------------------------------ the bias

// The boundaries, one or more a lane, so that the bucket of a uniform distance is
// a count over ballots.
struct Buckets {
    int b[kBucketsMax / 64];
    int n;               // boundaries
};

__device__ __forceinline__ Buckets load_buckets(const AttnArgs &A)
{
    Buckets B;
    B.n = A.bias ? A.buckets - 1 : 0;
#pragma unroll
    for (int t = 0; t < kBucketsMax / 64; t++) {
        const int j = 64 * t + lane_id();
        B.b[t] = j < B.n ? A.bnd[j] : INT32_MAX;
    }
    return B;
}

__device__ __forceinline__ int bucket_of(const Buckets &B, int x)
{
    int n = 0;
#pragma unroll
    for (int t = 0; t < kBucketsMax / 64; t++)
        if (64 * t < B.n) n += __popcll(__ballot(B.b[t] <= x));
    return uniform(min(n, B.n));
}

// --------------------------------------------------------------- key tiles

// What a stage of key rows brings besides K and V.
template <int KT>
struct KeyMeta {
    float out[KT];       // 0, or -inf where the key is masked or past the end
    int pos[KT];
    int lo[KT / 32], hi[KT / 32];   // range of positions of each 32 keys
};

// Loads keys [k0 + st .. + KT) of a sample that ends at k1 into LDS.  Masked keys
// and those past the end are zeros whatever the memory holds: their scores get -inf
// from the accumulator's initial value, and a probability of zero must not meet an
// infinity or NaN of V.
template <typename T, int DP, int KT>
__device__ __forceinline__ void stage_keys(const AttnArgs &A, int kvh, int64_t k0, int64_t k1, u32x4_t *lk,
                                           u32x4_t *lv, KeyMeta<KT> &M)
{
    using TL = Tile<T, DP>;
    const T *k = static_cast<const T *>(A.k) + kvh * A.kh, *v = static_cast<const T *>(A.v) + kvh * A.vh;
    const int t = threadIdx.x;
    static_assert(KT * TL::CH % kAttnThreads == 0, "whole chunks per thread");
#pragma unroll 8
    for (int i = t; i < KT * TL::CH; i += kAttnThreads) {
        const int r = i / TL::CH, c = i % TL::CH;
        const int64_t row = k0 + r;
        u32x4_t a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
        if (row < k1 && (!A.mask || *gp(A.mask + row))) {
            a = load_chunk(k + row * A.ks, c, A.dim, A.vec);
            b = load_chunk(v + row * A.vs, c, A.dim, A.vec);
        }
        lk[TL::at(r, c)] = a;
        lv[TL::at(r, c)] = b;
    }
    if (t < KT) {
        const int64_t row = k0 + t;
        const bool in = row < k1 && (!A.mask || *gp(A.mask + row));
        M.out[t] = in ? 0.f : -INFINITY;
        if (A.bias) {
            const int p = *gp(A.kp + (row < k1 ? row : k1 - 1));
            M.pos[t] = p;
            const int lo = min32(p), hi = max32(p);
            if ((t & 31) == 0) {
                M.lo[t / 32] = lo;
                M.hi[t / 32] = hi;
            }
        }
    }
}

// The range of stages a split takes of `n` stages.
__device__ __forceinline__ void split_range(int64_t n, int split, int splits, int64_t &a, int64_t &b)
{
    a = n * split / splits;
    b = n * (split + 1) / splits;
}

// The 32 query rows of a wavefront, one per lane & 31 (both halves hold the same).
struct Row {
    bool live;
    int64_t q;       // row of q
    int head, g;     // query head, its number inside the group
    int pos;
    int lo, hi;      // range of positions of the wavefront's rows
};

__device__ __forceinline__ Row query_row(const AttnArgs &A, const SegTile &s, int kvh, int64_t r0)
{
    Row R;
    const int64_t r = r0 + (lane_id() & 31);
    R.live = r < s.rows;
    const int64_t rc = R.live ? r : s.rows - 1;      // a row past the end repeats the last
    const int64_t i = rc / A.group;
    R.g = (int)(rc - i * A.group);
    R.q = s.base + i;
    R.head = kvh * A.group + R.g;
    R.pos = A.bias ? A.qp[R.q] : 0;
    R.lo = uniform(min32(R.pos));
    R.hi = uniform(max32(R.pos));
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

// Scores in units of log2: t_i = c s_i + bias * log2(e), returned as (s, c', b') with
// t_i = c' s_i + b'.  Where all pairs of the block fall in one bucket (most blocks:
// buckets widen with the distance) the bias is one number a row and costs nothing;
// otherwise each boundary inside the block's range is a compare and a select.
__device__ __forceinline__ void add_bias(const AttnArgs &A, const Buckets &B, const float *lb, const int *lbnd,
                                         const Row &R, const int *kpos, int klo, int khi, f32x16_t &s, float &c,
                                         float &b)
{
    c = A.c;
    b = 0.f;
    if (!A.bias) return;
    const int lo = bucket_of(B, sub_sat(R.lo, khi)), hi = bucket_of(B, sub_sat(R.hi, klo));
    const float *mine = lb + R.g;
    b = mine[lo * A.group];
    if (lo == hi) return;
    int x[16];
    f32x16_t t;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        x[i] = sub_sat(R.pos, kpos[block_key(i)]);
        t[i] = b;
    }
    for (int m = lo; m < hi; m++) {
        const int edge = lbnd[m];
        const float v = mine[(m + 1) * A.group];
#pragma unroll
        for (int i = 0; i < 16; i++) t[i] = x[i] >= edge ? v : t[i];
    }
#pragma unroll
    for (int i = 0; i < 16; i++) s[i] = fmaf(s[i], c, t[i]);
    c = 1.f;
    b = 0.f;
}

// The bias table of a key head's group, times log2(e), and the boundaries, in LDS.
__device__ __forceinline__ void stage_bias(const AttnArgs &A, int kvh, float *lb, int *lbnd)
{
    if (!A.bias) return;
    for (int i = threadIdx.x; i < A.buckets * A.group; i += kAttnThreads) {
        const int m = i / A.group, g = i - m * A.group;
        lb[i] = A.bias[(int64_t)m * A.heads + kvh * A.group + g] * kLog2e;
    }
    for (int i = threadIdx.x; i < A.buckets - 1; i += kAttnThreads) lbnd[i] = A.bnd[i];
}

// keys per stage of the kernels that walk the keys
template <typename T, int WM>
constexpr int key_stage()
{
    return WM == 4 ? (sizeof(T) == 2 ? 64 : 32) : 128;
}

// ------------------------------------------------------------------ forward

// WM = 4: the four wavefronts take 32 rows each and all keys.  WM = 1 (few rows per
// sample): one set of 32 rows, and each wavefront takes every fourth 32 keys; the
// four partial results meet in LDS.  With splits > 1 several workgroups share the
// keys of one set of rows and attn_join finishes.
template <typename T, int DP, int WM>
__global__ __launch_bounds__(kAttnThreads) void attn_forward(AttnArgs A)
{
    using TL = Tile<T, DP>;
    constexpr int KT = key_stage<T, WM>();
    constexpr int kTileWords = 2 * KT * TL::CH;
    constexpr int kJoinWords = WM == 1 ? 4 * 32 * DP / 4 : 0;
    __shared__ u32x4_t lds[kTileWords > kJoinWords ? kTileWords : kJoinWords];
    __shared__ KeyMeta<KT> M;
    __shared__ int lbnd[kBucketsMax];
    __shared__ float jm[4][32], jl[4][32];
    extern __shared__ float lb[];
    u32x4_t *lk = lds, *lv = lds + KT * TL::CH;

    const int64_t id = xcd_block(blockIdx.x, gridDim.x, 0);
    const int split = (int)(id % A.splits);
    const int64_t rest = id / A.splits;
    const int kvh = (int)(rest / A.tiles);
    const SegTile s = seg_find(A.qo, A.samples, A.nq, A.group, WM * 32, rest % A.tiles);
    if (s.row0 >= s.rows) return;
    const int lane = lane_id(), h = lane >> 5, w = uniform((int)(threadIdx.x >> 6));
    const int64_t r0 = s.row0 + (WM == 4 ? w * 32 : 0);
    const bool busy = r0 < s.rows;
    const bool nobody = s.seg == 0 || s.seg == A.samples + 1;
    const int64_t k0 = nobody ? 0 : seg_edge(A.ko, A.samples, A.nk, s.seg);
    const int64_t k1 = nobody ? 0 : seg_edge(A.ko, A.samples, A.nk, s.seg + 1);

    stage_bias(A, kvh, lb, lbnd);
    const Buckets B = load_buckets(A);
    const Row R = query_row(A, s, kvh, r0);
    Frag<T, DP> qf;
    load_frag<T, DP>(qf, static_cast<const T *>(A.q) + R.q * A.qs + R.head * A.qh, A.dim, A.vec, R.live);

    float m = -INFINITY, l = 0.f;
    f32x16_t o[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; d++) o[d] = f32x16_t{};
    bool any = false;

    int64_t st0, st1;
    split_range(k1 > k0 ? (k1 - k0 + KT - 1) / KT : 0, split, A.splits, st0, st1);
    for (int64_t st = st0; st < st1; st++) {
        const int64_t kb = k0 + st * KT;
        __syncthreads();
        stage_keys<T, DP, KT>(A, kvh, kb, k1, lk, lv, M);
        __syncthreads();
        if (!busy) continue;
        for (int sub = WM == 4 ? 0 : w; sub < (WM == 4 ? KT / 32 : w + 1); sub++) {
            if (kb + sub * 32 >= k1) break;
            f32x16_t sc = block_order(M.out + sub * 32);
            any |= __ballot(M.out[sub * 32 + (lane & 31)] == 0.f) != 0;
            products<T, DP>(sc, lk, sub * 32, qf);
            float c, b;
            add_bias(A, B, lb, lbnd, R, M.pos + sub * 32, M.lo[sub], M.hi[sub], sc, c, b);
            float top = sc[0];
#pragma unroll
            for (int i = 1; i < 16; i++) top = fmaxf(top, sc[i]);
            top = both_halves_max(fmaf(top, c, b));
            if (__ballot(top > m)) {
                const float mn = fmaxf(m, top);
                const float alpha = exp2_fast(m - (mn == -INFINITY ? 0.f : mn));
                m = mn;
                l *= alpha;
#pragma unroll
                for (int d = 0; d < DP / 32; d++)
#pragma unroll
                    for (int i = 0; i < 16; i++) o[d][i] *= alpha;
            }
            const float base = b - (m == -INFINITY ? 0.f : m);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 16; i++) {
                sc[i] = exp2_fast(fmaf(sc[i], c, base));
                sum += sc[i];
            }
            l += sum;
            const typename Mma<T>::Pack p = Mma<T>::pack(sc);
#pragma unroll
            for (int d = 0; d < DP / 32; d++) Mma<T>::template transposed<DP>(o[d], lv, sub * 32, d, p);
        }
    }
    l = both_halves_sum(l);
    if (!any) {            // no key at all: zero, also where q is not finite
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int d = 0; d < DP / 32; d++) o[d] = f32x16_t{};
    }

    if (WM == 1) {
        // the four wavefronts' parts of the same rows, scaled to a common maximum
        float *lo = reinterpret_cast<float *>(lds);
        __syncthreads();
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
            for (int i = 0; i < 16; i++) lo[(w * DP + 32 * d + block_key(i)) * 32 + (lane & 31)] = o[d][i] * f;
        __syncthreads();
        // wavefront w finishes the 8 (i >> 2) groups of d with i >> 2 == w
        m = mt;
        l = lt;
        float r[DP / 32][4];
#pragma unroll
        for (int d = 0; d < DP / 32; d++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int row = 32 * d + 8 * w + 4 * h + e;
                float x = 0.f;
#pragma unroll
                for (int u = 0; u < 4; u++) x += lo[(u * DP + row) * 32 + (lane & 31)];
                r[d][e] = x;
            }
        if (!R.live) return;
        const int64_t row = R.q * A.heads + R.head;
        if (A.splits > 1) {
            const int64_t at = (int64_t)split * A.nq * A.heads + row;
#pragma unroll
            for (int d = 0; d < DP / 32; d++)
#pragma unroll
                for (int e = 0; e < 4; e++) A.part[at * DP + 32 * d + 8 * w + 4 * h + e] = r[d][e];
            if (w == 0 && h == 0) {
                A.part_ml[2 * at] = m;
                A.part_ml[2 * at + 1] = l;
            }
            return;
        }
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
        T *out = static_cast<T *>(A.out) + row * A.dim;
#pragma unroll
        for (int d = 0; d < DP / 32; d++) {
            const int col = 32 * d + 8 * w + 4 * h;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = r[d][e] * inv;
            if (col + 4 <= A.dim && A.dim % 4 == 0) Mma<T>::store4(out + col, v);
            else
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (col + e < A.dim) Mma<T>::store1(out + col + e, v[e]);
        }
        if (w == 0 && h == 0 && A.lse) A.lse[row] = l > 0.f || l != l ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
        return;
    }

    if (!R.live || !busy) return;
    const int64_t row = R.q * A.heads + R.head;
    if (A.splits > 1) {
        const int64_t at = (int64_t)split * A.nq * A.heads + row;
#pragma unroll
        for (int d = 0; d < DP / 32; d++)
#pragma unroll
            for (int i = 0; i < 16; i++) A.part[at * DP + 32 * d + block_key(i)] = o[d][i];
        if (h == 0) {
            A.part_ml[2 * at] = m;
            A.part_ml[2 * at + 1] = l;
        }
        return;
    }
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    T *out = static_cast<T *>(A.out) + row * A.dim;
#pragma unroll
    for (int d = 0; d < DP / 32; d++)
#pragma unroll
        for (int g = 0; g < 4; g++) {
            const int col = 32 * d + 8 * g + 4 * h;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = o[d][4 * g + e] * inv;
            if (col + 4 <= A.dim && A.dim % 4 == 0) Mma<T>::store4(out + col, v);
            else
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (col + e < A.dim) Mma<T>::store1(out + col + e, v[e]);
        }
    if (h == 0 && A.lse) A.lse[row] = l > 0.f || l != l ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

// Joins the splits of a row: a wavefront per (row, head), a lane per element.
template <typename T, int DP>
__global__ __launch_bounds__(kAttnThreads) void attn_join(AttnArgs A)
{
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), n = A.nq * A.heads;
    if (row >= n) return;
    const int lane = lane_id();
    float m = -INFINITY;
    for (int u = 0; u < A.splits; u++) m = fmaxf(m, A.part_ml[2 * (u * n + row)]);
    const float mb = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[(DP + 63) / 64] = {};
    for (int u = 0; u < A.splits; u++) {
        const float f = exp2_fast(A.part_ml[2 * (u * n + row)] - mb);
        l += A.part_ml[2 * (u * n + row) + 1] * f;
#pragma unroll
        for (int e = 0; e < (DP + 63) / 64; e++)
            if (64 * e + lane < DP) o[e] += A.part[(u * n + row) * DP + 64 * e + lane] * f;
    }
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    T *out = static_cast<T *>(A.out) + row * A.dim;
#pragma unroll
    for (int e = 0; e < (DP + 63) / 64; e++)
        if (64 * e + lane < A.dim) Mma<T>::store1(out + 64 * e + lane, o[e] * inv);
    if (lane == 0 && A.lse) A.lse[row] = l > 0.f || l != l ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

// ------------------------------------------------------- backward: queries

// dq_i = scale (sum_j p_ij dP_ij k_j - delta_i sum_j p_ij k_j) with
// delta_i = sum_j p_ij dP_ij, all three sums in one pass over the keys.  Taking delta
// from the probabilities that the gradients use (and not from the output, which was
// rounded) costs a fourth product and makes the gradients of a row's scores add up
// to zero in fp32: the bias gradient is a sum of those over many rows and would
// otherwise drown in the rounding of the output.
template <typename T, int DP, int WM>
__global__ __launch_bounds__(kAttnThreads) void attn_backward_q(AttnArgs A)
{
    using TL = Tile<T, DP>;
    constexpr int KT = key_stage<T, WM>();
    constexpr int kTileWords = 2 * KT * TL::CH;
    constexpr int kJoinWords = WM == 1 ? 4 * 32 * DP / 4 : 0;
    __shared__ u32x4_t lds[kTileWords > kJoinWords ? kTileWords : kJoinWords];
    __shared__ KeyMeta<KT> M;
    __shared__ int lbnd[kBucketsMax];
    __shared__ float jd[4][32];
    extern __shared__ float lb[];
    u32x4_t *lk = lds, *lv = lds + KT * TL::CH;

    const int64_t id = xcd_block(blockIdx.x, gridDim.x, 0);
    const int split = (int)(id % A.splits);
    const int64_t rest = id / A.splits;
    const int kvh = (int)(rest / A.tiles);
    const SegTile s = seg_find(A.qo, A.samples, A.nq, A.group, WM * 32, rest % A.tiles);
    if (s.row0 >= s.rows) return;
    const int lane = lane_id(), h = lane >> 5, w = uniform((int)(threadIdx.x >> 6));
    const int64_t r0 = s.row0 + (WM == 4 ? w * 32 : 0);
    const bool busy = r0 < s.rows;
    const bool nobody = s.seg == 0 || s.seg == A.samples + 1;
    const int64_t k0 = nobody ? 0 : seg_edge(A.ko, A.samples, A.nk, s.seg);
    const int64_t k1 = nobody ? 0 : seg_edge(A.ko, A.samples, A.nk, s.seg + 1);

    stage_bias(A, kvh, lb, lbnd);
    const Buckets B = load_buckets(A);
    const Row R = query_row(A, s, kvh, r0);
    const int64_t row = R.q * A.heads + R.head;
    Frag<T, DP> qf, df;
    load_frag<T, DP>(qf, static_cast<const T *>(A.q) + R.q * A.qs + R.head * A.qh, A.dim, A.vec, R.live);
    load_frag<T, DP>(df, static_cast<const T *>(A.dout) + R.q * A.ds + R.head * A.dh, A.dim, A.vec, R.live);
    // a row without keys has lse = -inf: exp2(score - inf) keeps its weights zero
    float lse = R.live ? A.lse[row] * kLog2e : INFINITY;
    if (lse == -INFINITY) lse = INFINITY;

    float delta = 0.f;
    f32x16_t x[DP / 32], y[DP / 32];       // sum p dP k, sum p k
#pragma unroll
    for (int d = 0; d < DP / 32; d++) x[d] = y[d] = f32x16_t{};

    int64_t st0, st1;
    split_range(k1 > k0 ? (k1 - k0 + KT - 1) / KT : 0, split, A.splits, st0, st1);
    for (int64_t st = st0; st < st1; st++) {
        const int64_t kb = k0 + st * KT;
        __syncthreads();
        stage_keys<T, DP, KT>(A, kvh, kb, k1, lk, lv, M);
        __syncthreads();
        if (!busy) continue;
        for (int sub = WM == 4 ? 0 : w; sub < (WM == 4 ? KT / 32 : w + 1); sub++) {
            if (kb + sub * 32 >= k1) break;
            f32x16_t sc = block_order(M.out + sub * 32), dp = f32x16_t{};
            products<T, DP>(sc, lk, sub * 32, qf);
            products<T, DP>(dp, lv, sub * 32, df);
            float c, b;
            add_bias(A, B, lb, lbnd, R, M.pos + sub * 32, M.lo[sub], M.hi[sub], sc, c, b);
            b -= lse;
#pragma unroll
            for (int i = 0; i < 16; i++) {
                sc[i] = exp2_fast(fmaf(sc[i], c, b));
                dp[i] *= sc[i];
                delta += dp[i];
            }
            const typename Mma<T>::Pack p = Mma<T>::pack(sc), pd = Mma<T>::pack(dp);
#pragma unroll
            for (int d = 0; d < DP / 32; d++) {
                Mma<T>::template transposed<DP>(x[d], lk, sub * 32, d, pd);
                Mma<T>::template transposed<DP>(y[d], lk, sub * 32, d, p);
            }
        }
    }
    delta = both_halves_sum(delta);
    T *dq = static_cast<T *>(A.dq) + row * A.dim;
    if (WM == 1) {
        float *lo = reinterpret_cast<float *>(lds);
        float r[2][DP / 32][4];
        __syncthreads();
        if (h == 0) jd[w][lane & 31] = delta;
#pragma unroll
        for (int k = 0; k < 2; k++) {
            if (k) __syncthreads();
#pragma unroll
            for (int d = 0; d < DP / 32; d++)
#pragma unroll
                for (int i = 0; i < 16; i++)
                    lo[(w * DP + 32 * d + block_key(i)) * 32 + (lane & 31)] = k ? y[d][i] : x[d][i];
            __syncthreads();
#pragma unroll
            for (int d = 0; d < DP / 32; d++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    float z = 0.f;
#pragma unroll
                    for (int u = 0; u < 4; u++) z += lo[(u * DP + 32 * d + 8 * w + 4 * h + e) * 32 + (lane & 31)];
                    r[k][d][e] = z;
                }
        }
        delta = (jd[0][lane & 31] + jd[1][lane & 31]) + (jd[2][lane & 31] + jd[3][lane & 31]);
        if (!R.live) return;
        if (A.splits > 1) {
            const int64_t at = (int64_t)split * A.nq * A.heads + row;
#pragma unroll
            for (int d = 0; d < DP / 32; d++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    A.part[2 * at * DP + 32 * d + 8 * w + 4 * h + e] = r[0][d][e];
                    A.part[(2 * at + 1) * DP + 32 * d + 8 * w + 4 * h + e] = r[1][d][e];
                }
            if (w == 0 && h == 0) A.part_ml[at] = delta;
            return;
        }
#pragma unroll
        for (int d = 0; d < DP / 32; d++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int col = 32 * d + 8 * w + 4 * h + e;
                if (col < A.dim) Mma<T>::store1(dq + col, A.scale * (r[0][d][e] - delta * r[1][d][e]));
            }
        if (w == 0 && h == 0) A.delta[row] = delta;
        return;
    }
    if (!R.live || !busy) return;
    if (A.splits > 1) {
        const int64_t at = (int64_t)split * A.nq * A.heads + row;
#pragma unroll
        for (int d = 0; d < DP / 32; d++)
#pragma unroll
            for (int i = 0; i < 16; i++) {
                A.part[2 * at * DP + 32 * d + block_key(i)] = x[d][i];
                A.part[(2 * at + 1) * DP + 32 * d + block_key(i)] = y[d][i];
            }
        if (h == 0) A.part_ml[at] = delta;
        return;
    }
#pragma unroll
    for (int d = 0; d < DP / 32; d++)
#pragma unroll
        for (int g = 0; g < 4; g++) {
            const int col = 32 * d + 8 * g + 4 * h;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = A.scale * (x[d][4 * g + e] - delta * y[d][4 * g + e]);
            if (col + 4 <= A.dim && A.dim % 4 == 0) Mma<T>::store4(dq + col, v);
            else
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (col + e < A.dim) Mma<T>::store1(dq + col + e, v[e]);
        }
    if (h == 0) A.delta[row] = delta;
}

template <typename T, int DP>
__global__ __launch_bounds__(kAttnThreads) void attn_join_q(AttnArgs A)
{
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), n = A.nq * A.heads;
    if (row >= n) return;
    const int lane = lane_id();
    float delta = 0.f, x[(DP + 63) / 64] = {}, y[(DP + 63) / 64] = {};
    for (int u = 0; u < A.splits; u++) {
        delta += A.part_ml[u * n + row];
#pragma unroll
        for (int e = 0; e < (DP + 63) / 64; e++)
            if (64 * e + lane < DP) {
                x[e] += A.part[2 * (u * n + row) * DP + 64 * e + lane];
                y[e] += A.part[(2 * (u * n + row) + 1) * DP + 64 * e + lane];
            }
    }
    T *dq = static_cast<T *>(A.dq) + row * A.dim;
#pragma unroll
    for (int e = 0; e < (DP + 63) / 64; e++)
        if (64 * e + lane < A.dim) Mma<T>::store1(dq + 64 * e + lane, A.scale * (x[e] - delta * y[e]));
    if (lane == 0) A.delta[row] = delta;
}

// ---------------------------------------------------------- backward: keys

// query rows per stage
template <typename T, int DP>
constexpr int query_stage()
{
    return 32;
}

// A workgroup owns 128 keys of one key head, 32 a wavefront (one per lane & 31), K
// and V in registers, and walks all query rows of the sample, one head of the group
// after the other: dk and dv need no sum across workgroups.
template <typename T, int DP>
__global__ __launch_bounds__(kAttnThreads) void attn_backward_k(AttnArgs A)
{
    using TL = Tile<T, DP>;
    constexpr int QT = query_stage<T, DP>();
    __shared__ u32x4_t lq[QT * TL::CH], ld[QT * TL::CH];
    __shared__ float first[QT], ndelta[QT];    // - lse / c (or -inf), - delta
    __shared__ int qpos[QT], qlo[QT / 32], qhi[QT / 32];
    __shared__ int lbnd[kBucketsMax];
    __shared__ float acc[4][kBucketsMax];
    extern __shared__ float lb[];

    const int64_t id = xcd_block(blockIdx.x, gridDim.x, 0);
    const int kvh = (int)(id / A.tiles);
    const int64_t tile = id % A.tiles;
    const SegTile s = seg_find(A.ko, A.samples, A.nk, 1, 128, tile);
    const bool idle = s.row0 >= s.rows;
    const int lane = lane_id(), h = lane >> 5, w = uniform((int)(threadIdx.x >> 6));
    const bool nobody = s.seg == 0 || s.seg == A.samples + 1;
    int64_t q0 = nobody || idle ? 0 : seg_edge(A.qo, A.samples, A.nq, s.seg);
    int64_t q1 = nobody || idle ? 0 : seg_edge(A.qo, A.samples, A.nq, s.seg + 1);
    if (idle && !A.dbias_part) return;

    stage_bias(A, kvh, lb, lbnd);
    for (int i = threadIdx.x; i < 4 * kBucketsMax; i += kAttnThreads) (&acc[0][0])[i] = 0.f;
    const Buckets B = load_buckets(A);
    const int64_t r = s.row0 + 32 * w + (lane & 31);
    const bool in = r < s.rows;
    const int64_t key = s.base + (in ? r : s.rows - 1);
    const bool busy = !idle && s.row0 + 32 * w < s.rows;
    const bool live = in && !idle && (!A.mask || A.mask[key]);
    int kpos = 0, klo = 0, khi = 0;
    if (A.bias && !idle) {
        kpos = A.kp[key];
        klo = uniform(min32(kpos));
        khi = uniform(max32(kpos));
    }
    Frag<T, DP> kf, vf;
    load_frag<T, DP>(kf, static_cast<const T *>(A.k) + (live ? key * A.ks + kvh * A.kh : 0), A.dim, A.vec, live);
    load_frag<T, DP>(vf, static_cast<const T *>(A.v) + (live ? key * A.vs + kvh * A.vh : 0), A.dim, A.vec, live);

    f32x16_t dk[DP / 32], dv[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; d++) dk[d] = dv[d] = f32x16_t{};

    for (int g = 0; g < A.group; g++) {
        const int head = kvh * A.group + g;
        const T *q = static_cast<const T *>(A.q) + head * A.qh, *dout = static_cast<const T *>(A.dout) + head * A.dh;
        for (int64_t qb = q0; qb < q1; qb += QT) {
            __syncthreads();
            for (int i = threadIdx.x; i < QT * TL::CH; i += kAttnThreads) {
                const int rr = i / TL::CH, c = i % TL::CH;
                u32x4_t a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
                if (qb + rr < q1) {
                    a = load_chunk(q + (qb + rr) * A.qs, c, A.dim, A.vec);
                    b = load_chunk(dout + (qb + rr) * A.ds, c, A.dim, A.vec);
                }
                lq[TL::at(rr, c)] = a;
                ld[TL::at(rr, c)] = b;
            }
            if (threadIdx.x < QT) {
                const int t = threadIdx.x;
                const bool there = qb + t < q1;
                const int64_t row = (qb + t) * A.heads + head;
                const float lse = there ? A.lse[row] * kLog2e : -INFINITY;
                first[t] = lse == -INFINITY ? -INFINITY : -lse / A.c;
                ndelta[t] = there ? -A.delta[row] : 0.f;
                if (A.bias) {
                    const int p = A.qp[there ? qb + t : q1 - 1];
                    qpos[t] = p;
                    const int lo = min32(p), hi = max32(p);
                    if ((t & 31) == 0) {
                        qlo[t / 32] = lo;
                        qhi[t / 32] = hi;
                    }
                }
            }
            __syncthreads();
            if (!busy) continue;
#pragma unroll
            for (int sub = 0; sub < QT / 32; sub++) {
                if (qb + sub * 32 >= q1) break;
                f32x16_t sc = block_order(first + sub * 32), dp = block_order(ndelta + sub * 32);
                products<T, DP>(sc, lq, sub * 32, kf);
                products<T, DP>(dp, ld, sub * 32, vf);
                float b = live ? 0.f : -INFINITY, c = A.c;
                int lo = 0, hi = 0, x[16];
                if (A.bias) {
                    lo = bucket_of(B, sub_sat(qlo[sub], khi));
                    hi = bucket_of(B, sub_sat(qhi[sub], klo));
                    b += lb[lo * A.group + g];
                    if (lo != hi) {
                        f32x16_t t;
                        for (int i = 0; i < 16; i++) {
                            x[i] = sub_sat(qpos[sub * 32 + block_key(i)], kpos);
                            t[i] = b;
                        }
                        for (int m = lo; m < hi; m++) {
                            const int edge = lbnd[m];
                            const float v = live ? lb[(m + 1) * A.group + g] : -INFINITY;
#pragma unroll
                            for (int i = 0; i < 16; i++) t[i] = x[i] >= edge ? v : t[i];
                        }
#pragma unroll
                        for (int i = 0; i < 16; i++) sc[i] = fmaf(sc[i], c, t[i]);
                        c = 1.f;
                        b = 0.f;
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    sc[i] = exp2_fast(fmaf(sc[i], c, b));
                    dp[i] *= sc[i];
                }
                const typename Mma<T>::Pack p = Mma<T>::pack(sc), ds = Mma<T>::pack(dp);
#pragma unroll
                for (int d = 0; d < DP / 32; d++) {
                    Mma<T>::template transposed<DP>(dv[d], ld, sub * 32, d, p);
                    Mma<T>::template transposed<DP>(dk[d], lq, sub * 32, d, ds);
                }
                if (A.dbias_part) {
                    for (int m = lo; m <= hi; m++) {
                        float sum = 0.f;
                        if (m < hi) {
                            const int edge = lbnd[m];
#pragma unroll
                            for (int i = 0; i < 16; i++) {
                                const bool below = x[i] < edge;
                                sum += below ? dp[i] : 0.f;
                                dp[i] = below ? 0.f : dp[i];
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; i++) sum += dp[i];
                        }
                        sum = wave_sum(sum);
                        if (lane == 0) acc[w][m] += sum;
                    }
                }
            }
        }
        if (A.dbias_part) {
            __syncthreads();
            float *to = A.dbias_part + (tile * A.heads + head) * A.buckets;
            for (int m = threadIdx.x; m < A.buckets; m += kAttnThreads) {
                to[m] = (acc[0][m] + acc[1][m]) + (acc[2][m] + acc[3][m]);
                acc[0][m] = acc[1][m] = acc[2][m] = acc[3][m] = 0.f;
            }
            __syncthreads();
        }
    }
    if (!in || idle || !A.dk) return;
    T *pk = static_cast<T *>(A.dk) + (key * A.kv_heads + kvh) * A.dim;
    T *pv = static_cast<T *>(A.dv) + (key * A.kv_heads + kvh) * A.dim;
#pragma unroll
    for (int d = 0; d < DP / 32; d++)
#pragma unroll
        for (int g = 0; g < 4; g++) {
            const int col = 32 * d + 8 * g + 4 * h;
            float a[4], b[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                a[e] = A.scale * dk[d][4 * g + e];
                b[e] = dv[d][4 * g + e];
            }
            if (col + 4 <= A.dim && A.dim % 4 == 0) {
                Mma<T>::store4(pk + col, a);
                Mma<T>::store4(pv + col, b);
            } else
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (col + e < A.dim) {
                        Mma<T>::store1(pk + col + e, a[e]);
                        Mma<T>::store1(pv + col + e, b[e]);
                    }
        }
}

// dbias[m, head] = sum of the workgroups' parts, in a fixed order: a workgroup per
// (head, 64 buckets), four tiles side by side
__global__ __launch_bounds__(kAttnThreads) void attn_join_bias(AttnArgs A, float *dbias)
{
    __shared__ float part[4][64];
    const int head = blockIdx.x, lane = lane_id(), w = threadIdx.x >> 6;
    const int m = blockIdx.y * 64 + lane;
    float sum = 0.f;
    if (m < A.buckets)
        for (int64_t t = w; t < A.tiles; t += 4) sum += A.dbias_part[(t * A.heads + head) * A.buckets + m];
    part[w][lane] = sum;
    __syncthreads();
    if (w == 0 && m < A.buckets)
        dbias[(int64_t)m * A.heads + head] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
}

}  // namespace emb

using namespace emb;

namespace {

size_t pad256(size_t x) { return (x + 255) & ~size_t(255); }

// How the kernels that walk the keys are cut: 32 or 128 query rows a workgroup, and
// the number of workgroups that share the keys of one set of rows.
struct AttnPlan {
    int wm, splits;
    int64_t tiles, key_tiles;
};

AttnPlan attn_plan(const emb_attention *a)
{
    AttnPlan p{};
    const int group = a->heads / a->kv_heads;
    const int64_t rows = a->n_q * group, samples = a->samples > 0 ? a->samples : 1;
    p.wm = rows / samples > 64 ? 4 : 1;
    p.tiles = seg_tiles(a->n_q, a->samples, group, 32 * p.wm);
    const int64_t sets = (rows / (32 * p.wm) > std::min<int64_t>(samples, a->n_q) ? rows / (32 * p.wm)
                                                                                  : std::min<int64_t>(samples, a->n_q)) *
                         a->kv_heads;
    const int64_t stages = a->n_k / samples / 128;     // of the average sample
    int64_t s = sets > 0 ? (1024 + sets - 1) / sets : 1;
    s = std::min<int64_t>(s, std::max<int64_t>(1, stages / 2));
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(s, 128));
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
        n += pad256(rows * padded_dim(a->dim) * 8) + pad256(rows * 4);
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
    if (a->n_q >= (int64_t(1) << 31) - 1 || a->n_k >= (int64_t(1) << 31) - 1 || a->samples >= (1 << 30))
        return fail(EMB_ERR_UNSUPPORTED, "attention: n_q and n_k must be < 2^31 - 1 and samples < 2^30 (int32 offsets)");
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

// rows that can be read in 16-byte pieces: whole pieces per row, every row aligned
bool wide_rows(const void *p, int64_t stride, int64_t head_stride, int dim, size_t el)
{
    return aligned(p, 16) && stride * el % 16 == 0 && head_stride * el % 16 == 0 && dim * el % 16 == 0;
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
    A.nq = a->n_q;
    A.nk = a->n_k;
    A.samples = a->samples;
    A.heads = a->heads;
    A.kv_heads = a->kv_heads;
    A.group = a->heads / a->kv_heads;
    A.dim = a->dim;
    A.buckets = a->buckets;
    A.scale = a->scale;
    A.c = a->scale * kLog2e;
    A.vec = wide_rows(a->q, a->q_stride, a->q_head_stride, a->dim, el) &&
            wide_rows(a->k, a->k_stride, a->k_head_stride, a->dim, el) &&
            wide_rows(a->v, a->v_stride, a->v_head_stride, a->dim, el);
    A.splits = p.splits;
    A.tiles = p.tiles;
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
    const dim3 grid((unsigned)(p.tiles * A.kv_heads * p.splits)), block(kAttnThreads);
    if (p.wm == 4) hipLaunchKernelGGL((attn_forward<T, DP, 4>), grid, block, lds, st, A);
    else hipLaunchKernelGGL((attn_forward<T, DP, 1>), grid, block, lds, st, A);
    if (p.splits > 1)
        hipLaunchKernelGGL((attn_join<T, DP>), dim3((unsigned)((A.nq * A.heads + 3) / 4)), block, 0, st, A);
    return launched("attention forward");
}

template <typename T, int DP>
emb_status backward_run(const AttnArgs &A0, const AttnPlan &p, float *dbias, hipStream_t st)
{
    AttnArgs A = A0;
    const size_t lds = (size_t)A.buckets * A.group * 4;
    const dim3 block(kAttnThreads);
    if (A.nq) {
        const dim3 grid((unsigned)(p.tiles * A.kv_heads * p.splits));
        if (p.wm == 4) hipLaunchKernelGGL((attn_backward_q<T, DP, 4>), grid, block, lds, st, A);
        else hipLaunchKernelGGL((attn_backward_q<T, DP, 1>), grid, block, lds, st, A);
        if (p.splits > 1)
            hipLaunchKernelGGL((attn_join_q<T, DP>), dim3((unsigned)((A.nq * A.heads + 3) / 4)), block, 0, st, A);
    }
    A.tiles = p.key_tiles;
    if (A.dk || dbias)
        hipLaunchKernelGGL((attn_backward_k<T, DP>), dim3((unsigned)(p.key_tiles * A.kv_heads)), block, lds, st, A);
    if (dbias)
        hipLaunchKernelGGL(attn_join_bias, dim3((unsigned)A.heads, (unsigned)((A.buckets + 63) / 64)), block, 0, st, A,
                           dbias);
    return launched("attention backward");
}

bool grid_fits(const emb_attention *a, const AttnPlan &p)
{
    const double most = 2147483647.0;
    return (double)p.tiles * a->kv_heads * p.splits <= most && (double)p.key_tiles * a->kv_heads <= most &&
           (double)a->n_q * a->heads / 4 + 1 <= most;
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

extern "C" emb_status emb_attention_forward(const emb_attention *a, void *out, float *lse, void *workspace,
                                            size_t workspace_bytes, void *stream)
{
    emb_status s = attn_check(a);
    if (s == EMB_OK) s = attn_pointers(a);
    if (s != EMB_OK) return s;
    if (a->n_q == 0) return EMB_OK;
    const size_t el = a->dtype == EMB_BF16 ? 2 : 4;
    if (!out || !aligned(out, a->dim % 4 == 0 ? 4 * el : el) || !aligned(lse, 4))
        return fail(EMB_ERR_INVALID_ARG, "attention: out must be given and aligned to four elements");
    const AttnPlan p = attn_plan(a);
    if (!grid_fits(a, p)) return fail(EMB_ERR_UNSUPPORTED, "attention: more than 2^31 - 1 workgroups");
    const size_t need = forward_workspace(a, p);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return fail(EMB_ERR_WORKSPACE, "attention: the workspace is smaller than the query returned, or not 256-byte aligned");
    AttnArgs A = attn_args(a, p);
    A.out = out;
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

extern "C" emb_status emb_attention_backward(const emb_attention *a, const float *lse, const void *dout,
                                             int64_t dout_stride, int64_t dout_head_stride, void *dq, void *dk,
                                             void *dv, float *dbias, void *workspace, size_t workspace_bytes,
                                             void *stream)
{
    emb_status s = attn_check(a);
    if (s == EMB_OK) s = attn_pointers(a);
    if (s != EMB_OK) return s;
    const size_t el = a->dtype == EMB_BF16 ? 2 : 4;
    const size_t al = a->dim % 4 == 0 ? 4 * el : el;
    if (a->n_q && (!lse || !dout || !dq))
        return fail(EMB_ERR_INVALID_ARG, "attention: lse, dout and dq must be given");
    if (!dk != !dv) return fail(EMB_ERR_INVALID_ARG, "attention: dk and dv are given together");
    if (dbias && !a->buckets) return fail(EMB_ERR_INVALID_ARG, "attention: dbias without a bias");
    if (!aligned(dout, el) || !aligned(dq, al) || !aligned(dk, al) || !aligned(dv, al) || !aligned(lse, 4) ||
        !aligned(dbias, 4))
        return fail(EMB_ERR_INVALID_ARG, "attention: gradients must be aligned to four elements");
    if (dout_stride < 0 || dout_head_stride < 0) return fail(EMB_ERR_INVALID_ARG, "attention: strides must be >= 0");
    const AttnPlan p = attn_plan(a);
    if (!grid_fits(a, p)) return fail(EMB_ERR_UNSUPPORTED, "attention: more than 2^31 - 1 workgroups");
    const size_t need = backward_workspace(a, p);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return fail(EMB_ERR_WORKSPACE, "attention: the workspace is smaller than the query returned, or not 256-byte aligned");
    AttnArgs A = attn_args(a, p);
    A.dout = dout;
    A.ds = dout_stride;
    A.dh = dout_head_stride;
    A.vec = A.vec && wide_rows(dout, dout_stride, dout_head_stride, a->dim, el);
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
        ws += pad256(rows * padded_dim(a->dim) * 8);
        A.part_ml = reinterpret_cast<float *>(ws);
        ws += pad256(rows * 4);
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
