// delta.hip -- the gated delta rule over jagged sequences, a recurrence whose state is a
// matrix S [dk, dv] per sample and head,
//   a_t = sigmoid(gate_t), b_t = sigmoid(beta_t),
//   u_t = b_t (v_t - a_t S_(t-1)^T k_t),  S_t = a_t S_(t-1) + k_t u_t^T,  o_t = scale S_t^T q_t,
// its backward pass and its one-step form.
//
// 32 rows are taken together (a chunk).  With S the state before them, G_i the product of
// a_1 .. a_i, e_ij = G_i / G_j, W_i = G_32 / G_i and row vectors stacked to matrices Q, K, V, U:
//   M_ij = b_i e_ij k_i.k_j (j < i),  N = (I + M)^-1,  P_ij = scale e_ij q_i.k_j (j <= i)
//   U = N (b (V - G (K S))),  O = scale G (Q S) + P U,  S' = G_32 S + K^T (W U)
// and backwards, with E the gradient of S' (and dS that of S):
//   dU = P^T dO + W (K E),  Z = N^T dU,  dV = b Z,
//   dS = G_32 E + Q^T (scale G dO) - K^T (b G Z)
//   D_ij = scale e_ij dO_i.u_j (j <= i),  B_ij = -b_i e_ij Z_i.u_j (j < i)
//   dQ = scale G (dO S^T) + D K
//   dK = W (U E^T) - b G (Z S^T) + D^T Q + (B + B^T) K
//   dbeta_i = (1 - b_i) Z_i.u_i
// The gradient of log a_t is what every e_ij, G_i and W_j that a_t is a factor of brings:
// with H_ij = D_ij q_i.k_j + B_ij k_i.k_j,
//   sum of H_ij over i >= t > j,  + sum over i >= t of (scale G_i q_i.(S dO_i) - b_i G_i k_i.(S Z_i)),
//   + sum over j < t of W_j k_j.(E u_j),  + G_32 <E, S>;   dgate_t = (1 - a_t) times that.
//
// Four kernels: delta_prepare (all chunks side by side) makes N, P and the scalars,
// delta_scan walks the chunks of a sample, delta_back walks them backwards, delta_grads
// (all chunks side by side) makes the gradients that need both sides' states.  The walks
// take 16 columns of the state per wavefront, which never meet one another.
//
// What passes between them costs more than the rows themselves: what bounds the four is bytes,
// then a walk's chain of dependent products.  bf16, 287434 rows in 256 samples, 4 heads of
// 64 x 64: prepare 142 us (0.64 GB, 4.5 TB/s), scan 229 us (0.93 GB, 4.0 TB/s).  With
// gradients, 68548 rows in 64 samples, 4 heads of 128 x 128: prepare 63 us, scan 316 us and back
// 342 us (1.07 GB each; the longest of 256 walks on 256 CUs is twice the mean), grads 525 us
// (1.75 GB, 3.3 TB/s).
//
// All products run on the matrix cores, the walks' in blocks of 16 x 16 (lane & 15 a column,
// register i of quarter g = lane >> 4 row 4 g + i), the others' in 32 x 32 (lane & 31 a column,
// register i of half h = lane >> 5 row kk(i, h) = 8 (i >> 2) + 4 h + (i & 3)), which is also how
// the next product takes its second operand if its contraction runs in that order.  The state
// is fp32.  What enters a product is cut into bf16 parts, the first rounded from the value,
// the next from what is left of it: inputs in bf16 are one part, all else three (24 bits).
// Products of parts whose bits lie below the last part's are left out.  What passes between the
// kernels is fp32 or three parts, so that a bf16 call computes what an fp32 call does from the same
// numbers, to the bit, and rounds it once (what only bf16 outputs are made of in two parts, 16 bits:
// 0.3 % of a bf16 output's elements one step away).
#include <string>

#include "sequence.h"

namespace emb {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr int kCut = 32;                 // rows of a chunk
constexpr int kSpan = 1024;              // rows of a segment of a cut sample
constexpr int kDeltaDim = 128;           // largest head size
// the scalars of a chunk and head, in floats: what the walks take, and what the gradients take too
constexpr int kScB = 0, kScBG = 32, kScG = 64, kScW = 96, kScEnd = 127, kScWalk = 128, kScHi = 128, kScLo = 160,
              kScKept = 192, kScalars = 256;

struct DeltaArgs {
    const void *q, *k, *v, *gate, *beta;            // rows and heads any stride apart (elements)
    int64_t qs, qh, ks, kh, vs, vh, gs, bs;
    const int32_t *off;
    const uint8_t *mask;
    const float *state;
    int32_t n, samples, key_heads, heads, group, dk, dv, slices;
    float scale;
    char *rec;                 // records of (tile, head): N, P, scalars
    int64_t rec_size;
    void *s0, *u;              // saved for the backward, of (tile, head): the state before in fp32, and U, as operands
    int32_t *order;            // samples from the longest on, or NULL: as they are
    int32_t ranks;             // workgroups of delta_prepare that make it
    int32_t cut;               // samples are cut into segments
    int32_t moves_back;        // ... whose transposed matrices are wanted too
    uint16_t *moves;           // of (segment, head): what it does to a state, in parts (and transposed)
    int64_t move_size;
    float *starts;             // of (segment, head): what it adds, then the state it begins with
    void *o;
    float *last;
    const void *dout;
    int64_t ds, dh;            // strides of dout
    const float *dlast;
    void *e, *z;               // E as s0, Z as u
    void *dq, *dk_, *dv_, *dgate, *dbeta;
    float *dstate;
    int32_t vec, ovec;         // dq and dk rows move in pieces of 4; o and dv rows in 16 bytes
};

// parts of the inputs and of what is made of them
template <typename T>
constexpr int kIn = sizeof(T) == 2 ? 1 : 3;
constexpr int kParts = 3;

__device__ __forceinline__ constexpr int kk0(int i) { return 8 * (i >> 2) + (i & 3); }   // + 4 h

template <int N>
struct Part {
    u32x4_t p[N];
};

// 8 values as bf16 parts
template <int N>
__device__ __forceinline__ Part<N> split8(const float *v)
{
    Part<N> r;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        float a = v[2 * j], b = v[2 * j + 1];
#pragma unroll
        for (int i = 0; i < N; i++) {
            const uint32_t w = bf16x2_rne(a, b);
            r.p[i][j] = w;
            a -= bf16_lo(w);
            b -= bf16_hi(w);
        }
    }
    return r;
}

// acc += A B over 16 elements of the contraction, parts of orders below ORD, the smallest first
template <int ORD, int NA, int NB>
__device__ __forceinline__ void mm(f32x16_t &acc, const Part<NA> &a, const Part<NB> &b)
{
#pragma unroll
    for (int s = ORD - 1; s >= 0; s--)
#pragma unroll
        for (int i = 0; i < NA; i++)
            if (s - i >= 0 && s - i < NB)
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a.p[i]),
                                                              __builtin_bit_cast(bf16x8_t, b.p[s - i]), acc, 0, 0, 0);
}

template <int ORD, int NA, int NB>
__device__ __forceinline__ void mm(f32x4_t &acc, const Part<NA> &a, const Part<NB> &b)
{
#pragma unroll
    for (int s = ORD - 1; s >= 0; s--)
#pragma unroll
        for (int i = 0; i < NA; i++)
            if (s - i >= 0 && s - i < NB)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.p[i]),
                                                              __builtin_bit_cast(bf16x8_t, b.p[s - i]), acc, 0, 0, 0);
}

// ... over 16 elements, the first or the second half of b's
template <int ORD, int NA, int NB>
__device__ __forceinline__ void mm_half(f32x4_t &acc, const u32x2_t (&a)[NA], const Part<NB> &b, int half)
{
#pragma unroll
    for (int s = ORD - 1; s >= 0; s--)
#pragma unroll
        for (int i = 0; i < NA; i++)
            if (s - i >= 0 && s - i < NB) {
                const u32x4_t w = b.p[s - i];
                acc = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(
                    __builtin_bit_cast(s16x4_t, a[i]), __builtin_bit_cast(s16x4_t, u32x2_t{w[2 * half], w[2 * half + 1]}), acc, 0, 0, 0);
            }
}

// 32 rows x 16 columns of a walk: t[a][i] of quarter g is row 16 a + 4 g + i
struct Block {
    f32x4_t t[2];
};

__device__ __forceinline__ Block zero_block() { return Block{{{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}}; }

// ... as a second operand, its rows contracted in the order 16 (e >> 2) + 4 g + (e & 3)
template <int N>
__device__ __forceinline__ Part<N> operand(const Block &x)
{
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = x.t[e >> 2][e & 3];
    return split8<N>(v);
}

__device__ __forceinline__ f32x16_t zero16()
{
    f32x16_t z;
#pragma unroll
    for (int i = 0; i < 16; i++) z[i] = 0.f;
    return z;
}

// registers 8 kc .. 8 kc + 7 of a block as a second operand
template <int N>
__device__ __forceinline__ Part<N> operand(const f32x16_t &x, int kc)
{
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = x[8 * kc + e];
    return split8<N>(v);
}

__device__ __forceinline__ u32x4_t buf16(__amdgpu_buffer_rsrc_t r, uint32_t at)
{
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, 0, 0));
}

template <typename T>
struct Row;
// Eight elements in memory as a lane's part of an operand (at kNowhere: zeros), and single ones.
template <>
struct Row<uint16_t> {
    typedef Part<1> Op;
    static __device__ __forceinline__ Op eight(__amdgpu_buffer_rsrc_t r, uint32_t at) { return Op{{buf16(r, at)}}; }
    static __device__ __forceinline__ void put4(uint16_t *p, const float *v)
    {
        *gp(reinterpret_cast<u32x2_t *>(p)) = u32x2_t{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
    }
    static __device__ __forceinline__ void put1(uint16_t *p, float v) { *gp(p) = bf16_rne(v); }
    static __device__ __forceinline__ float get1(const uint16_t *p) { return bf16_lo((uint32_t)*gp(p)); }
};
template <>
struct Row<float> {
    typedef Part<3> Op;
    static __device__ __forceinline__ Op eight(__amdgpu_buffer_rsrc_t r, uint32_t at)
    {
        float f[8];
        const u32x4_t a = buf16(r, at), b = buf16(r, at + 16);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            f[j] = __uint_as_float(a[j]);
            f[4 + j] = __uint_as_float(b[j]);
        }
        return split8<3>(f);
    }
    static __device__ __forceinline__ void put4(float *p, const float *v)
    {
        *gp(reinterpret_cast<f32x4_t *>(p)) = f32x4_t{v[0], v[1], v[2], v[3]};
    }
    static __device__ __forceinline__ void put1(float *p, float v) { *gp(p) = v; }
    static __device__ __forceinline__ float get1(const float *p) { return *gp(p); }
};

// a buffer from an address that is the same in every lane
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p, int64_t elements)
{
    return row_buffer(static_cast<const T *>(p) + elements, 0, 0x7FFFFFFF);
}

// A record: the scalars of the walks, N - I and P in their parts, the other scalars.  The matrices
// are triangular.  A part is rows 16 .. in a KB, a row's 4 pieces of 16 bytes side by side, piece g
// (columns 4 g .. and 16 + 4 g ..) of row r at g ^ (r >> 2), see Lane, and columns .. 15 of the
// other rows in 512 bytes, pieces of 8 bytes, g of row r at g ^ (r >> 3) * 2 (so that 32 lanes that
// read 16 rows meet every bank once).  10 KB; with whole matrices it would be 13.
constexpr int kMatrix = 3 * 512;
struct Rec {
    static constexpr int sc = 0, n = kScWalk * 4, p = n + kParts * kMatrix, more = p + kParts * kMatrix, size = more + (kScalars - kScWalk) * 4;
};
__device__ __forceinline__ uint32_t matrix_above(int row, int quad) { return 1024 + (row * 4 + (quad ^ (row >> 3) * 2)) * 8; }
__device__ __forceinline__ uint32_t matrix_below(int row, int piece) { return (row * 4 + (piece ^ (row >> 2))) * 16; }

// e^(hi + lo): the product with log2(e) to more bits than one rounding
__device__ __forceinline__ float exp_of(float hi, float lo)
{
    const float t = hi * kLog2e;
    const float r = fmaf(hi, kLog2e, -t) + fmaf(hi, 1.9259629911266175e-8f, lo * kLog2e);
    return exp2_fast(t) * fmaf(r, kLn2, 1.f);
}

// sum of a value and the other half's
__device__ __forceinline__ float both(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// where a sample's chunks are numbered from (the tiles of seg_find)
__device__ __forceinline__ int first_tile(int base, int sample) { return base / kCut + sample + 1; }

// ----------------------------------------------------------------- prepare

// Walks begin in the order of their lengths, the longest first, since what begins last ends last
// (256 samples of 200..2000 rows, the scan: 289 us in the samples' own order, 232 so).  A lane counts the samples
// that come before its own; wavefronts beside the chunks' do it.  Lengths from 2^20 on count as one.
constexpr int kRanked = 1024;
__device__ __forceinline__ void delta_order(const DeltaArgs &A, int block)
{
    const int l = lane_id(), own = 64 * block + l;
    auto key = [&](int s) {                              // no two are equal
        const int rows = seg_edge(A.off, A.samples, A.n, s + 2) - seg_edge(A.off, A.samples, A.n, s + 1);
        return s < A.samples ? min(max(rows, 0), (1 << 20) - 1) * kRanked + kRanked - 1 - s : -1;
    };
    const int mine = key(own);
    int before = 0, next = key(l);
    for (int s0 = 0; s0 < A.samples; s0 += 64) {
        const int theirs = next;
        next = key(s0 + 64 + l);
#pragma unroll
        for (int j = 0; j < 64; j++) before += __builtin_amdgcn_readlane(theirs, j) > mine ? 1 : 0;
    }
    if (own < A.samples) *gp(A.order + before) = own;
}

// A chunk's scalars, P and N, a wavefront a chunk and head.  Sums of log a are fp64: they reach
// 32 x 200, and what e^ is taken of are their differences.  N comes by forward substitution, a
// column a lane, which keeps fp32's accuracy where keys repeat (powers of M do not).
template <typename T, int KT>
__global__ __launch_bounds__(64) void delta_prepare(DeltaArgs A)
{
    constexpr int kPitch = 36;
    __shared__ __attribute__((aligned(16))) float lds[32 * kPitch];
    __shared__ __attribute__((aligned(16))) float sc[kScalars];
    const int tile = (int)blockIdx.x - A.ranks, head = blockIdx.y, key = head / A.group;
    if (tile < 0) {
        if (head == 0) delta_order(A, blockIdx.x);
        return;
    }
    const int l = lane_id(), c = l & 31, h = l >> 5;
    const SegTile s = seg_find<kCut>(A.off, A.n, nullptr, 0, A.samples, 1, tile);
    if (s.row0 >= s.rows) return;
    const int left = min(s.rows - s.row0, kCut);
    const int64_t row = (int64_t)s.base + s.row0;
    if (s.seg == 0 || s.seg == A.samples + 1) {          // rows of no sample
        for (int r = 0; r < left; r++)
            for (int x = l; x < A.dv; x += 64)
                Row<T>::put1(static_cast<T *>(A.o) + ((row + r) * A.heads + head) * A.dv + x, 0.f);
        return;
    }
    const bool valid = c < left;
    const bool keep = valid && (!A.mask || *gp(A.mask + row + c));
    const uint32_t kept = (uint32_t)__ballot(keep);
    // the rows' scalars; log a is at least -200, where a is zero in fp32
    float la = 0.f, b = 0.f;
    if (keep) {
        const float g = Row<T>::get1(static_cast<const T *>(A.gate) + (row + c) * A.gs + head);
        const float x = Row<T>::get1(static_cast<const T *>(A.beta) + (row + c) * A.bs + head);
        la = (g < 0.f ? g : g != g ? g : 0.f) - log1pf(expf(-fabsf(g)));
        if (la < -200.f) la = -200.f;
        b = 1.f / (1.f + expf(-x));
    }
    double sum = la;                                     // of log a up to here
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const double x = __shfl_up(sum, d, 32);
        if (c >= d) sum += x;
    }
    const double whole = __shfl(sum, 31, 32);
    const float hi = (float)sum, lo = (float)(sum - hi);
    const float G = exp_of(hi, lo);
    const double after = whole - sum;
    const float ahi = (float)after, W = exp_of(ahi, (float)(after - ahi));
    if (h == 0) {
        sc[kScB + c] = b;
        sc[kScBG + c] = b * G;
        sc[kScG + c] = A.scale * G;
        sc[kScW + c] = c == 31 ? G : W;                  // W of the last row is 1: G_32 is there
        sc[kScHi + c] = hi;
        sc[kScLo + c] = lo;
        if (c == 31) sc[kScKept] = __uint_as_float(kept);
    }
    wave_sync();
    char *rec = A.rec + ((int64_t)tile * A.heads + head) * A.rec_size;
    // what only the gradients take is left for them alone
    if (l < kScWalk / 4 || A.s0 || l == kScKept / 4)
        *gp(reinterpret_cast<f32x4_t *>(rec + (l < kScWalk / 4 ? Rec::sc : Rec::more - kScWalk * 4)) + l) =
            *reinterpret_cast<const f32x4_t *>(sc + 4 * l);

    const auto qb = buffer<T>(A.q, row * A.qs + key * A.qh), kb = buffer<T>(A.k, row * A.ks + key * A.kh);
    const uint32_t qat = keep ? (uint32_t)(c * A.qs * sizeof(T)) : kNowhere;
    const uint32_t kat = keep ? (uint32_t)(c * A.ks * sizeof(T)) : kNowhere;
    f32x16_t kk = zero16(), kq = zero16();                     // a lane's row, the others in registers
#pragma unroll
    for (int x = 0; x < 2 * KT; x++) {
        const uint32_t at = (uint32_t)((16 * x + 8 * h) * sizeof(T));
        const auto K = Row<T>::eight(kb, kat + at), Q = Row<T>::eight(qb, qat + at);
        mm<kIn<T>>(kk, K, K);
        mm<kIn<T>>(kq, K, Q);                                  // k_j.q_i, lane i
    }
    // P and M as rows of i, in LDS, and from there into the record
    float m[16];
#pragma unroll
    for (int g4 = 0; g4 < 4; g4++) {
        const int j0 = 8 * g4 + 4 * h;
        const f32x4_t ghi = *reinterpret_cast<const f32x4_t *>(sc + kScHi + j0);
        const f32x4_t glo = *reinterpret_cast<const f32x4_t *>(sc + kScLo + j0);
        f32x4_t p;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int j = j0 + e, r = 4 * g4 + e;
            const float d = j <= c ? exp_of(hi - ghi[e], lo - glo[e]) : 0.f;
            p[e] = j <= c ? A.scale * d * kq[r] : 0.f;
            m[r] = j < c ? b * d * kk[r] : 0.f;
        }
        *reinterpret_cast<f32x4_t *>(lds + c * kPitch + j0) = p;
    }
    auto leave = [&](int at) {                           // the matrix in LDS into the record
        const int row = l & 15, g = l >> 4;
#pragma unroll
        for (int a = 0; a < 2; a++) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const f32x4_t x = *reinterpret_cast<const f32x4_t *>(lds + (16 * a + row) * kPitch + 4 * e + 4 * g);
#pragma unroll
                for (int i = 0; i < 4; i++) f[e + i] = x[i];
            }
            const Part<kParts> p = split8<kParts>(f);
#pragma unroll
            for (int i = 0; i < kParts; i++) {
                char *to = rec + at + i * kMatrix;
                if (a) *gp(reinterpret_cast<u32x4_t *>(to + matrix_below(row, g))) = p.p[i];
                else *gp(reinterpret_cast<u32x2_t *>(to + matrix_above(row, g))) = u32x2_t{p.p[i][0], p.p[i][1]};
            }
        }
    };
    wave_sync();
    leave(Rec::p);
    wave_sync();
#pragma unroll
    for (int g4 = 0; g4 < 4; g4++)
        *reinterpret_cast<f32x4_t *>(lds + c * kPitch + 8 * g4 + 4 * h) =
            f32x4_t{m[4 * g4], m[4 * g4 + 1], m[4 * g4 + 2], m[4 * g4 + 3]};
    wave_sync();
    // N by forward substitution, a column a lane: n_i = [i = c] - sum over j < i of M_ij n_j
    float nn[32];
#pragma unroll
    for (int i = 0; i < 32; i++) {
        float x = i == c ? 1.f : 0.f;
#pragma unroll
        for (int j4 = 0; j4 < (i + 3) / 4; j4++) {
            const f32x4_t mi = *reinterpret_cast<const f32x4_t *>(lds + i * kPitch + 4 * j4);
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (4 * j4 + e < i) x = fmaf(-mi[e], nn[4 * j4 + e], x);
        }
        nn[i] = x;
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < 16; i++) lds[(16 * h + i) * kPitch + c] = 16 * h + i == c ? 0.f : h ? nn[16 + i] : nn[i];
    wave_sync();
    leave(Rec::n);
}

// ------------------------------------------------------------ chunks in LDS

// For the gradients the rows of a chunk lie in LDS as operands of 32 rows: 1 KB holds 16 bytes of 32 rows, lane l = 32 h + r
// has row r; bf16: piece x has elements 16 x + 8 h + 0 .. 7, fp32: pieces 2 x and 2 x + 1 have
// the first and the last four of these.  They arrive there asynchronously.
template <typename T>
struct Lds {
    static constexpr int R = sizeof(T) / 2;              // pieces of 16 elements
    static constexpr int kRows = 1024 * R;               // bytes of 32 rows x 16 elements

    // 16 x + 8 h + 0 .. 7 of the lane's row
    static __device__ __forceinline__ typename Row<T>::Op rows(uint32_t at, int x)
    {
        const uint32_t mine = at + 16 * lane_id() + x * kRows;
        if constexpr (R == 1) return typename Row<T>::Op{{lds_read<u32x4_t>(mine)}};
        else {
            float f[8];
            const u32x4_t a = lds_read<u32x4_t>(mine), b = lds_read<u32x4_t>(mine + 1024);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                f[j] = __uint_as_float(a[j]);
                f[4 + j] = __uint_as_float(b[j]);
            }
            return split8<3>(f);
        }
    }
    // Where the lane's part of a column begins: element (lane & 31) of 32, of four rows in a row
    // from row 4 h.
    static __device__ __forceinline__ uint32_t column()
    {
        const int l = lane_id(), h = l >> 5;
        if constexpr (R == 1) {
            // sixteen lanes read 4 rows of 16 elements and get a column of 4 each
            const int q = l & 3, r = 4 * h + ((l & 15) >> 2);
            return (l >> 4 & 1) * 1024 + ((q >> 1) * 32 + r) * 16 + (q & 1) * 8;
        } else {
            const int c = l & 31;
            return ((c >> 4) * 2 + (c >> 2 & 1)) * 1024 + ((c >> 3 & 1) * 32 + 4 * h) * 16 + (c & 3) * 4;
        }
    }
    // the rows transposed as an operand: rows 16 kc + kk(e, h) of column 32 t + lane & 31
    static __device__ __forceinline__ typename Row<T>::Op turned(uint32_t at, uint32_t column, int t, int kc)
    {
        if constexpr (R == 1) {
            u32x4_t w;
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4_t *)(uintptr_t)(at + column + t * 2 * kRows + (16 * kc + 8 * j) * 16));
                const u32x2_t u = __builtin_bit_cast(u32x2_t, v);
                w[2 * j] = u[0];
                w[2 * j + 1] = u[1];
            }
            return typename Row<T>::Op{{w}};
        } else {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; e++)
                f[e] = lds_read<float>(at + column + t * 2 * kRows + (16 * kc + 8 * (e >> 2) + (e & 3)) * 16);
            return split8<3>(f);
        }
    }
    // elements 32 t + 8 g4 + 4 h + 0 .. 3 of the lane's row
    static __device__ __forceinline__ void own(uint32_t at, int t, int g4, float *f)
    {
        const int l = lane_id(), h = l >> 5;
        const uint32_t from = at + (2 * t + (g4 >> 1)) * kRows + ((g4 & 1) * 32 + (l & 31)) * 16;
        if constexpr (R == 1) {
            const u32x2_t w = lds_read<u32x2_t>(from + 8 * h);
#pragma unroll
            for (int j = 0; j < 2; j++) {
                f[2 * j] = bf16_lo(w[j]);
                f[2 * j + 1] = bf16_hi(w[j]);
            }
        } else {
            const u32x4_t w = lds_read<u32x4_t>(from + 1024 * h);
#pragma unroll
            for (int j = 0; j < 4; j++) f[j] = __uint_as_float(w[j]);
        }
    }
};

// Wavefront `wave` of `waves` brings every waves-th piece of 1 KB: rows of `pieces` KB (`at`: the
// lane's row and half in bytes, or kNowhere) into operands, ...
template <typename T>
__device__ __forceinline__ void bring_rows(i32x4_t rsrc, uint32_t at, uint32_t to, int pieces, int wave, int waves)
{
    constexpr int R = Lds<T>::R;
#pragma unroll 1
    for (int p = wave; p < pieces * R; p += waves)
        load_to_lds(rsrc, to + p * 1024, at, R == 1 ? p * 32 : (p >> 1) * 64 + (p & 1) * 16);
}
// ... or what lies so already
__device__ __forceinline__ void bring_flat(i32x4_t rsrc, uint32_t to, int pieces, int wave, int waves)
{
#pragma unroll 1
    for (int p = wave; p < pieces; p += waves)
        load_to_lds(rsrc, (uint32_t)uniform((int)(to + p * 1024)), 16 * lane_id(), (uint32_t)uniform(p * 1024));
}

// the operand of a record in LDS
template <int N>
__device__ __forceinline__ Part<N> staged(uint32_t at, int index)
{
    Part<N> r;
#pragma unroll
    for (int i = 0; i < N; i++) r.p[i] = lds_read<u32x4_t>(at + (index * N + i) * 1024 + 16 * lane_id());
    return r;
}

// what this wavefront brought has arrived, then what the workgroup did
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// ... of a wavefront that brings nothing, whose stores nobody in the workgroup waits for
__device__ __forceinline__ void meet_others() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1; }

template <typename T>
__device__ __forceinline__ uint32_t row_at(uint32_t kept, int64_t stride)
{
    const int l = lane_id(), r = l & 31;
    return kept >> r & 1 ? (uint32_t)(r * stride * sizeof(T)) + (l >> 5) * 8 * (uint32_t)sizeof(T) : kNowhere;
}

// For the walks the rows of a chunk lie in LDS as 16 rows x 32 elements a KB (fp32: two KB, the
// first and the last four of every eight), a row's 4 pieces of 16 bytes side by side, piece g
// of row r at g ^ (r >> 2): then neither 16 lanes that take a piece of 16 rows nor 16 that take
// a column of 4 rows meet on a bank.
template <typename T>
struct Lane {
    static constexpr int R = sizeof(T) / 2, kTile = 1024 * R;      // bytes of 16 rows x 32 elements
    uint32_t rows, keys;     // where the lane's first operands begin: rows, and columns for the state's update
    uint32_t above, turned, turned_above;   // ... and rows and columns of a record's matrix
    int r, q;                // (bf16) its row and quad of a column

    __device__ __forceinline__ Lane()
    {
        const int l = lane_id(), g = l >> 4, i = l & 15;
        rows = (i * 4 + (g ^ (i >> 2))) * 16;
        r = 4 * g + (i >> 2);
        q = i & 3;
        above = matrix_above(i, g);
        turned_above = matrix_above(r, q);
        // State rows are kept so that the registers of a block meet rows of K and Q as they lie in
        // memory: t[a][i] of quarter g is row 8 g + 4 a + i.
        turned = matrix_below(r, q);
        if (R == 1) keys = turned;
        else keys = (16 * g + ((i >> 2) ^ g)) * 16 + (i & 3) * 4;
    }
    // rows 16 a + lane & 15, elements 32 x + 8 g + 0 .. 7
    __device__ __forceinline__ typename Row<T>::Op row(uint32_t at, int x, int a) const
    {
        const uint32_t from = at + rows + (x * 2 + a) * kTile;
        if constexpr (R == 1) return typename Row<T>::Op{{lds_read<u32x4_t>(from)}};
        else {
            float f[8];
            const u32x4_t lo = lds_read<u32x4_t>(from), hi = lds_read<u32x4_t>(from + 1024);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                f[j] = __uint_as_float(lo[j]);
                f[4 + j] = __uint_as_float(hi[j]);
            }
            return split8<3>(f);
        }
    }
    // row 8 (i >> 2) + 4 a + (i & 3), i = lane & 15, of block x of the transposed rows
    __device__ __forceinline__ typename Row<T>::Op column(uint32_t at, int x, int a) const
    {
        if constexpr (R == 1) {
            u32x4_t w;
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const u32x2_t v = __builtin_bit_cast(u32x2_t, column4(at + keys + (x * 2 + j) * kTile + 8 * a));
                w[2 * j] = v[0];
                w[2 * j + 1] = v[1];
            }
            return typename Row<T>::Op{{w}};
        } else {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; e++) f[e] = lds_read<float>(at + keys + (x * 2 + (e >> 2)) * kTile + a * 1024 + (e & 3) * 64);
            return split8<3>(f);
        }
    }
    // elements 32 x + 8 g + 0 .. 7 of row r, for the lanes of quarter g, and element c
    static __device__ __forceinline__ void eight(uint32_t at, int r, int x, float *f)
    {
        const int g = lane_id() >> 4, i = r & 15;
        const uint32_t from = at + (x * 2 + (r >> 4)) * kTile + (i * 4 + (g ^ (i >> 2))) * 16;
        const u32x4_t a = lds_read<u32x4_t>(from);
        if constexpr (R == 1) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                f[2 * j] = bf16_lo(a[j]);
                f[2 * j + 1] = bf16_hi(a[j]);
            }
        } else {
            const u32x4_t b = lds_read<u32x4_t>(from + 1024);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                f[j] = __uint_as_float(a[j]);
                f[4 + j] = __uint_as_float(b[j]);
            }
        }
    }
    static __device__ __forceinline__ float one(uint32_t at, int r, int c)
    {
        const int i = r & 15, e = c & 7;
        const uint32_t from = at + ((c >> 5) * 2 + (r >> 4)) * kTile + (i * 4 + ((c >> 3 & 3) ^ (i >> 2))) * 16;
        if constexpr (R == 1) return bf16_lo((uint32_t)lds_read<uint16_t>(from + 2 * e));
        else return lds_read<float>(from + (e >> 2) * 1024 + (e & 3) * 4);
    }
    // sixteen lanes read 4 rows of 16 elements and get a column of 4 each
    static __device__ __forceinline__ s16x4_t column4(uint32_t at)
    {
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t *)(uintptr_t)at);
    }
    // acc += a record's matrix times x, and the matrix transposed times x
    template <int ORD, int N, int NB>
    __device__ __forceinline__ void matrix(Block &acc, uint32_t at, const Part<NB> &x) const
    {
        u32x2_t upper[N];
        Part<N> lower;
#pragma unroll
        for (int i = 0; i < N; i++) {
            upper[i] = lds_read<u32x2_t>(at + above + i * kMatrix);
            lower.p[i] = lds_read<u32x4_t>(at + rows + i * kMatrix);
        }
        mm_half<ORD>(acc.t[0], upper, x, 0);
        mm<ORD>(acc.t[1], lower, x);
    }
    template <int ORD, int N, int NB>
    __device__ __forceinline__ void matrix_turned(Block &acc, uint32_t at, const Part<NB> &x) const
    {
        Part<N> left;
        u32x2_t right[N];
#pragma unroll
        for (int i = 0; i < N; i++) {
            const uint32_t from = at + i * kMatrix;
            const u32x2_t y = __builtin_bit_cast(u32x2_t, column4(from + turned_above)), z = __builtin_bit_cast(u32x2_t, column4(from + turned));
            left.p[i] = u32x4_t{y[0], y[1], z[0], z[1]};
            right[i] = __builtin_bit_cast(u32x2_t, column4(from + turned + 8));
        }
        mm<ORD>(acc.t[0], left, x);
        mm_half<ORD>(acc.t[1], right, x, 1);
    }
    // where columns 16 slice .. begin, and these as a block
    __device__ __forceinline__ uint32_t columns(int slice) const
    {
        const int l = lane_id(), g = l >> 4, i = l & 15, x = slice >> 1, odd = slice & 1;
        if (R == 1) return (r * 4 + ((2 * odd + (q >> 1)) ^ g)) * 16 + (q & 1) * 8 + x * 2 * kTile;
        const int c = 16 * odd + i;
        return (16 * g + ((c >> 3) ^ g)) * 16 + (c >> 2 & 1) * 1024 + (c & 3) * 4 + x * 2 * kTile;
    }
    __device__ __forceinline__ Block block(uint32_t at, uint32_t columns) const
    {
        Block b;
#pragma unroll
        for (int a = 0; a < 2; a++)
            if constexpr (R == 1) {
                const s16x4_t v = column4(at + columns + a * kTile);
#pragma unroll
                for (int e = 0; e < 4; e++) b.t[a][e] = __uint_as_float((uint32_t)(uint16_t)v[e] << 16);
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++) b.t[a][e] = lds_read<float>(at + columns + a * kTile + 64 * e);
            }
        return b;
    }
};

// Brings 32 rows of `blocks` x 32 elements into that order.
template <typename T>
__device__ __forceinline__ void bring_tiles(const T *from, int64_t stride, uint32_t kept, uint32_t to, int blocks)
{
    constexpr int R = sizeof(T) / 2;
    const i32x4_t rsrc = row_rsrc(from);
    const int l = lane_id(), r = l >> 2, g = (l & 3) ^ (l >> 4);
    const uint32_t at = (uint32_t)(r * stride * sizeof(T)) + g * 8 * (uint32_t)sizeof(T);
    const uint32_t first = kept >> r & 1 ? at : kNowhere;
    const uint32_t second = kept >> (16 + r) & 1 ? at + (uint32_t)(16 * stride * sizeof(T)) : kNowhere;
    for (int x = 0; x < blocks; x++)
#pragma unroll
        for (int a = 0; a < 2; a++)
#pragma unroll
            for (int j = 0; j < R; j++, to += 1024) load_to_lds(rsrc, to, a ? second : first, x * 32 * sizeof(T) + j * 16);
}

// a scalar for each of a block's rows, of a record in LDS
__device__ __forceinline__ Block row_scalars(uint32_t at)
{
    Block r;
#pragma unroll
    for (int a = 0; a < 2; a++) r.t[a] = lds_read<f32x4_t>(at + 64 * a + 16 * (lane_id() >> 4));
    return r;
}

// W: its last place in a record is G_32's
__device__ __forceinline__ Block row_weights(uint32_t sc)
{
    Block r = row_scalars(sc + 4 * kScW);
    if (lane_id() >> 4 == 3) r.t[1][3] = 1.f;
    return r;
}

// Blocks whose columns lie in lanes, turned into rows by a wavefront's own scratch: fill() puts
// rows r0 .. r0 + 3 of the lane's column, take() gets elements 8 h + 0 .. 7 of row lane & 31, as
// they are stored.
template <typename T>
struct Turn {
    static constexpr int R = sizeof(T) / 2, kBytes = R == 1 ? 16 * 72 : 32 * 17 * 4;
    u32x4_t w[R];

    static __device__ __forceinline__ void fill(uint32_t scratch, int r0, const f32x4_t &f)
    {
        const int c = lane_id() & 15;
        if constexpr (R == 1) lds_write(scratch + c * 72 + r0 * 2, u32x2_t{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3])});
        else
#pragma unroll
            for (int e = 0; e < 4; e++) lds_write(scratch + ((r0 + e) * 17 + c) * 4, f[e]);
    }
    __device__ __forceinline__ void take(uint32_t scratch)
    {
        const int l = lane_id(), h = l >> 5;
        if constexpr (R == 1) {
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4_t *)(uintptr_t)(
                        scratch + (8 * h + 4 * j + ((l & 15) >> 2)) * 72 + (16 * (l >> 4 & 1) + 4 * (l & 3)) * 2)));
                w[0][2 * j] = v[0];
                w[0][2 * j + 1] = v[1];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) w[e >> 2][e & 3] = lds_read<uint32_t>(scratch + ((l & 31) * 17 + 8 * h + e) * 4);
        }
    }
    __device__ __forceinline__ void turn(uint32_t scratch, const Block &b)
    {
        const int g = lane_id() >> 4;
        wave_sync();
#pragma unroll
        for (int a = 0; a < 2; a++) fill(scratch, 16 * a + 4 * g, b.t[a]);
        wave_sync();
        take(scratch);
    }
    // as operands for the gradients
    __device__ __forceinline__ void keep(char *to) const
    {
#pragma unroll
        for (int j = 0; j < R; j++) *gp(reinterpret_cast<u32x4_t *>(to + j * 1024) + lane_id()) = w[j];
    }
    // columns c .. (the lane's, at `to`) of its row, where it is there
    __device__ __forceinline__ void write(T *to, bool there, int c, int dv, bool vec) const
    {
        if (!there) return;
        constexpr int E = 16 / sizeof(T);                // elements of 16 bytes
#pragma unroll
        for (int j = 0; j < R; j++) {
            if (vec) {
                if (c + j * E < dv) *gp(reinterpret_cast<u32x4_t *>(to + j * E)) = w[j];
            } else {
#pragma unroll
                for (int e = 0; e < E; e++) {
                    const uint32_t x = w[j][e * sizeof(T) / 4];
                    if (c + j * E + e < dv) {
                        if constexpr (sizeof(T) == 2) *gp(to + j * E + e) = (uint16_t)(e & 1 ? x >> 16 : x);
                        else *gp(to + j * E + e) = __uint_as_float(x);
                    }
                }
            }
        }
    }
};

// ----------------------------------------------------------------- the walks

// Rows of one sample and head that a workgroup walks over: whole samples, or, where samples
// are cut, segments of kSpan rows.
struct Walk {
    int head, key, base, rows, tile0;
    int64_t matrix;          // number of the sample's and head's state
    int64_t part;            // number of the segment's and head's record (cut samples)
    bool any, first, last;
};

__device__ __forceinline__ Walk walk_of(const DeltaArgs &A)
{
    Walk w{};
    int sample;
    const int unit = (int)(blockIdx.x / (uint32_t)A.heads);
    w.head = (int)(blockIdx.x - (uint32_t)unit * (uint32_t)A.heads);
    w.key = w.head / A.group;
    if (A.cut) {
        const SegTile s = seg_find<kSpan>(A.off, A.n, nullptr, 0, A.samples, 1, unit);
        w.any = s.row0 < s.rows && s.seg != 0 && s.seg != A.samples + 1;
        sample = s.seg - 1;
        w.base = s.base + s.row0;
        w.rows = min(s.rows - s.row0, kSpan);
        w.first = s.row0 == 0;
        w.last = s.row0 + kSpan >= s.rows;
        w.tile0 = first_tile(s.base, sample) + s.row0 / kCut;
        w.part = (int64_t)unit * A.heads + w.head;
    } else {
        sample = A.order ? uniform(*gp(A.order + unit)) : unit;
        w.any = w.first = w.last = true;
        w.base = uniform(seg_edge(A.off, A.samples, A.n, sample + 1));
        w.rows = max(uniform(seg_edge(A.off, A.samples, A.n, sample + 2)) - w.base, 0);
        w.tile0 = first_tile(w.base, sample);
    }
    w.matrix = (int64_t)sample * A.heads + w.head;
    return w;
}

// a wavefront's 16 columns of a state [dk, dv] in memory: t[a][i] of block x, quarter g is row
// 32 x + 8 g + 4 a + i
// the lane's place in a state; columns behind the last are out of its buffer, as are rows
__device__ __forceinline__ uint32_t state_lane(int dv, int col)
{
    return col < dv ? (uint32_t)(8 * (lane_id() >> 4) * dv + col) * 4 : kNowhere;
}
template <int KT>
__device__ __forceinline__ void state_read(Block (&S)[KT], const float *p, int dk, int dv, int col)
{
    const auto from = row_buffer(p, 0, p ? dk * dv * 4 : 0);
    const uint32_t at = state_lane(dv, col);
#pragma unroll
    for (int x = 0; x < KT; x++)
#pragma unroll
        for (int i = 0; i < 8; i++)
            S[x].t[i >> 2][i & 3] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(from, at + (32 * x + i) * dv * 4, 0, 0));
}
template <int KT>
__device__ __forceinline__ void state_write(const Block (&S)[KT], float *p, int dk, int dv, int col)
{
    const auto to = row_buffer(p, 0, dk * dv * 4);
    const uint32_t at = state_lane(dv, col);
#pragma unroll
    for (int x = 0; x < KT; x++)
#pragma unroll
        for (int i = 0; i < 8; i++)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[x].t[i >> 2][i & 3]), to, at + (32 * x + i) * dv * 4, 0, 0);
}

// a wavefront's scratch: for rows of T, and in training for the state's in fp32
template <typename T, bool TRAIN>
constexpr int kScratch = TRAIN ? Turn<float>::kBytes : Turn<T>::kBytes;
// A block's rows as the gradients read them, in fp32, 2 KB, and block x of the state.
__device__ __forceinline__ void rows_keep(uint32_t scratch, const Block &b, char *to)
{
    Turn<float> rows;
    rows.turn(scratch, b);
    rows.keep(to);
}
__device__ __forceinline__ void state_keep(uint32_t scratch, const Block &S, char *to, int x, int slices, int slice)
{
    const int g = lane_id() >> 4;
    Turn<float> rows;
    wave_sync();
#pragma unroll
    for (int a = 0; a < 2; a++) Turn<float>::fill(scratch, 8 * g + 4 * a, S.t[a]);
    wave_sync();
    rows.take(scratch);
    rows.keep(to + (x * slices + slice) * Lds<float>::kRows);
}

// A walk's workgroup.  A wavefront has 16 columns of the state, and one more brings the chunks, one
// ahead, and does nothing else.  SUM walks take no Q and no P.
template <typename T, int KT, bool SUM>
struct WalkLds {
    static constexpr int q = 2 * KT * Lane<T>::kTile, rec = SUM ? q : 2 * q, sc = rec + Rec::sc, n = rec + Rec::n,
                         p = rec + Rec::p, pieces = ((SUM ? Rec::p : Rec::more) + 1023) / 1024, v = rec + pieces * 1024;
    static __host__ __device__ constexpr int size(int slices) { return v + (slices + 1) / 2 * 2 * Lane<T>::kTile; }
};

// the bits of a chunk's rows that are kept (there, and not masked)
template <typename T>
__device__ __forceinline__ uint32_t kept_rows(const DeltaArgs &A, const Walk &w, int chunk)
{
    const int left = min(w.rows - chunk * kCut, kCut);
    if (chunk < 0 || left <= 0) return 0;
    const char *rec = A.rec + ((int64_t)(w.tile0 + chunk) * A.heads + w.head) * A.rec_size;
    return __float_as_uint(*gp(reinterpret_cast<const float *>(rec + Rec::more) + kScKept - kScWalk)) & low_bits(left);
}

// The wavefront that brings the chunks, in the order chunk(0), chunk(1), ... (steps of the walk);
// values: of v, or of the output's gradient
template <typename T, int KT, bool SUM, typename Chunk>
__device__ __forceinline__ void bring_chunks(const DeltaArgs &A, const Walk &w, int chunks, const Chunk &chunk, uint32_t at0,
                                             const void *values, int64_t vs, int64_t vh)
{
    typedef WalkLds<T, KT, SUM> L;
    auto bring = [&](int s, uint32_t kept) {
        const int64_t row = (int64_t)w.base + chunk(s) * kCut;
        const uint32_t to = at0 + (s & 1) * L::size(A.slices);
        bring_tiles<T>(static_cast<const T *>(A.k) + row * A.ks + w.key * A.kh, A.ks, kept, to, KT);
        if (!SUM) bring_tiles<T>(static_cast<const T *>(A.q) + row * A.qs + w.key * A.qh, A.qs, kept, to + L::q, KT);
        if (values) bring_tiles<T>(static_cast<const T *>(values) + row * vs + w.head * vh, vs, kept, to + L::v, (A.slices + 1) / 2);
        const i32x4_t rsrc = row_rsrc(A.rec + ((int64_t)(w.tile0 + chunk(s)) * A.heads + w.head) * A.rec_size);
#pragma unroll
        for (int p = 0; p < L::pieces; p++) load_to_lds(rsrc, to + L::rec + p * 1024, 16 * lane_id(), p * 1024);
    };
    if (!chunks) return;
    uint32_t kept = kept_rows<T>(A, w, chunk(0)), next = kept_rows<T>(A, w, chunks > 1 ? chunk(1) : -1);
    bring(0, kept);
    for (int s = 0; s < chunks; s++) {
        meet();
        kept = next;
        if (s + 1 < chunks) bring(s + 1, kept);
        next = kept_rows<T>(A, w, s + 2 < chunks ? chunk(s + 2) : -1);
    }
}

// Values that are not finite.  A chunk's matrices have zeros where a row has nothing of another,
// and zero times NaN or infinity is NaN: as products they would carry a row's NaN to rows before it.  A wavefront
// whose U (backward: Z) is not finite throughout takes that chunk and all behind it row by row, as the rule is
// written.
__device__ __forceinline__ bool any_spoiled(const Block &b)
{
    float x = 0.f;
#pragma unroll
    for (int a = 0; a < 2; a++)
#pragma unroll
        for (int e = 0; e < 4; e++) x = fmaf(b.t[a][e], 0.f, x);
    return __ballot(x != x) != 0;
}

// sum over the quarters, which share a column
__device__ __forceinline__ float quarters(float x)
{
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}

// a row's share in a block: row r of the lane's column
__device__ __forceinline__ void put_row(Block &b, int r, float x)
{
#pragma unroll
    for (int a = 0; a < 2; a++)
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (16 * a + 4 * (lane_id() >> 4) + e == r) b.t[a][e] = x;
}

template <typename T>
__device__ __forceinline__ float logistic_at(const void *p, int64_t at)
{
    return 1.f / (1.f + expf(-Row<T>::get1(static_cast<const T *>(p) + at)));
}

// f(row in the chunk, a, b) for a chunk's kept rows, from the first or from the last on
template <typename T, bool BACK, typename F>
__device__ __forceinline__ void by_rows(const DeltaArgs &A, const Walk &w, int chunk, const F &f)
{
    const uint32_t kept = kept_rows<T>(A, w, chunk);
#pragma unroll 1
    for (int i = 0; i < kCut; i++) {
        const int r = BACK ? kCut - 1 - i : i;
        if (!(kept >> r & 1)) continue;
        const int64_t row = (int64_t)w.base + chunk * kCut + r;
        f(r, logistic_at<T>(A.gate, row * A.gs + w.head), logistic_at<T>(A.beta, row * A.bs + w.head));
    }
}

// s = f(s, k) for the lane's numbers s of a state, k that of row r of K or Q (at `at`) there; rows of the
// state that are not there stay zeros
template <typename T, int KT, typename F>
__device__ __forceinline__ void state_rows(Block (&S)[KT], uint32_t at, int r, int dk, const F &f)
{
#pragma unroll
    for (int x = 0; x < KT; x++) {
        float k[8];
        Lane<T>::eight(at, r, x, k);
        int rows = dk - 32 * x - 8 * (lane_id() >> 4);
        asm volatile("" : "+v"(rows));                   // not made ahead of the loop over rows
#pragma unroll
        for (int i = 0; i < 8; i++) S[x].t[i >> 2][i & 3] = i < rows ? f(S[x].t[i >> 2][i & 3], k[i]) : S[x].t[i >> 2][i & 3];
    }
}

template <typename T, int KT>
__device__ __forceinline__ void scan_rows(const DeltaArgs &A, const Walk &w, int chunk, uint32_t at, int col, Block (&S)[KT],
                                          Block &U, Block &Y)
{
    typedef WalkLds<T, KT, false> L;
    U = Y = zero_block();
    by_rows<T, false>(A, w, chunk, [&](int r, float a, float b) {
        float held = 0.f, out = 0.f;
        state_rows<T>(S, at, r, A.dk, [&](float s, float k) {
            s *= a;
            held = fmaf(s, k, held);
            return s;
        });
        const float u = b * (Lane<T>::one(at + L::v, r, col) - quarters(held));
        state_rows<T>(S, at, r, A.dk, [&](float s, float k) { return fmaf(k, u, s); });
        state_rows<T>(S, at + L::q, r, A.dk, [&](float s, float q) {
            out = fmaf(s, q, out);
            return s;
        });
        put_row(U, r, u);
        put_row(Y, r, A.scale * quarters(out));
    });
}

template <typename T, int KT>
__device__ __forceinline__ void back_rows(const DeltaArgs &A, const Walk &w, int chunk, uint32_t at, int col, Block (&E)[KT],
                                          Block &Z, Block &dV)
{
    typedef WalkLds<T, KT, false> L;
    Z = dV = zero_block();
    by_rows<T, true>(A, w, chunk, [&](int r, float a, float b) {
        const float d = A.scale * Lane<T>::one(at + L::v, r, col);
        float z = 0.f;
        state_rows<T>(E, at + L::q, r, A.dk, [&](float e, float q) { return fmaf(q, d, e); });
        state_rows<T>(E, at, r, A.dk, [&](float e, float k) {
            z = fmaf(e, k, z);
            return e;
        });
        z = quarters(z);
        state_rows<T>(E, at, r, A.dk, [&](float e, float k) { return a * fmaf(-k, b * z, e); });
        put_row(Z, r, z);
        put_row(dV, r, b * z);
    });
}

// elements of a segment's matrix in its three parts
template <int KT>
constexpr int kMove = 3 * 1024 * KT * KT;

// Where element (row, col) of a segment's matrix lies, in bf16, the first of its 3 parts, which
// are 512 apart: KBs of 16 rows (one block of registers of a state) x 32 columns, first operands
// of delta_join, those of the same columns side by side.
template <int KT>
__device__ __forceinline__ int move_at(int row, int col)
{
    const int y = row >> 5, a = row >> 2 & 1, m = (row >> 3 & 3) * 4 + (row & 3);
    return (((col >> 5) * KT + y) * 2 + a) * 3 * 512 + ((col >> 3 & 3) * 16 + m) * 8 + (col & 7);
}

// Walks forward, a workgroup a sample and head.  Half the columns a workgroup, twice the workgroups,
// evened unequal samples out but read K, Q and records twice (with states kept in bf16, a step of
// training of 64 samples with 4 heads of 128: 764 us and 852 so, a long history forward 392 and 440).
// SUM: a segment's own part alone, what it adds (blockIdx.y 0) and what it does to the state, as a
// matrix (1: the walk without values from the identity).
template <typename T, int KT, bool TRAIN, bool SUM>
__global__ __launch_bounds__(576) void delta_scan(DeltaArgs A)
{
    typedef WalkLds<T, KT, SUM> L;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const Walk w = walk_of(A);
    if (!w.any) return;
    const bool values = !SUM || blockIdx.y == 0;
    const int slice = uniform((int)(threadIdx.x >> 6)), slices = values ? A.slices : 2 * KT;
    const int chunks = (w.rows + kCut - 1) / kCut;
    const uint32_t at0 = lds_address(lds);
    if (slice >= slices) {
        auto order = [](int s) { return s; };
        if (slice == slices) bring_chunks<T, KT, SUM>(A, w, chunks, order, at0, values ? A.v : nullptr, A.vs, A.vh);
        return;                                          // the rest: fewer columns of one kind than of the other
    }
    const int l = lane_id(), r = l & 31, c = 16 * slice + 8 * (l >> 5), col = 16 * slice + (l & 15);
    const uint32_t scratch = at0 + 2 * L::size(A.slices) + slice * kScratch<T, TRAIN>;
    const Lane<T> lane;
    const uint32_t columns = lane.columns(values ? slice : 0);

    Block S[KT];
    if (SUM) {
#pragma unroll
        for (int x = 0; x < KT; x++)
#pragma unroll
            for (int i = 0; i < 8; i++) S[x].t[i >> 2][i & 3] = !values && 32 * x + 8 * (l >> 4) + i == col ? 1.f : 0.f;
    } else
        state_read<KT>(S, A.cut ? A.starts + w.part * A.dk * A.dv : A.state ? A.state + w.matrix * A.dk * A.dv : nullptr, A.dk,
                       A.dv, col);
    // what leaves: the lane's piece of a row of o, of U and of the states, a chunk's step apart
    const int64_t ostep = (int64_t)kCut * A.heads * A.dv, ustep = (int64_t)A.heads * A.slices * 2048,
                  sstep = (int64_t)A.heads * KT * A.slices * Lds<float>::kRows;
    T *o = static_cast<T *>(A.o) + ((int64_t)(w.base + r) * A.heads + w.head) * A.dv + c;
    const int64_t number = (int64_t)w.tile0 * A.heads + w.head;
    char *u = static_cast<char *>(A.u) + (number * A.slices + slice) * 2048;
    char *states = static_cast<char *>(A.s0) + number * KT * A.slices * Lds<float>::kRows;
    auto leave = [&](int chunk, const Block &U, const Block &Y) {
        if (TRAIN) rows_keep(scratch, U, u);
        Turn<T> rows;
        rows.turn(scratch, Y);
        rows.write(o, r < w.rows - chunk * kCut, c, A.dv, A.ovec);
        o += ostep;
        u += ustep;
        states += sstep;
    };
    int i = 0;
    for (; i < chunks; i++) {
        meet_others();
        const uint32_t at = at0 + (i & 1) * L::size(A.slices), sc = at + L::sc;
        Block X = zero_block(), Y = zero_block(), V = zero_block();
#pragma unroll
        for (int x = 0; x < KT; x++) {
            const Part<kParts> sp = operand<kParts>(S[x]);
            if (TRAIN && !SUM) state_keep(scratch, S[x], states, x, A.slices, slice);
#pragma unroll
            for (int a = 0; a < 2; a++) {
                mm<kParts>(X.t[a], lane.row(at, x, a), sp);
                if (!SUM) mm<kParts>(Y.t[a], lane.row(at + L::q, x, a), sp);
            }
        }
        const Block b = row_scalars(sc + 4 * kScB), bg = row_scalars(sc + 4 * kScBG);
        if (values) V = lane.block(at + L::v, columns);
#pragma unroll
        for (int a = 0; a < 2; a++)
#pragma unroll
            for (int e = 0; e < 4; e++) X.t[a][e] = fmaf(b.t[a][e], V.t[a][e], -bg.t[a][e] * X.t[a][e]);
        const Part<kParts> xp = operand<kParts>(X);
        Block U = X;                                     // N is I and what the record has
        lane.template matrix<kParts, kParts>(U, at + L::n, xp);
        if (!SUM && __builtin_expect(any_spoiled(U), 0)) break;
        const Block wt = row_weights(sc);
        const float end = lds_read<float>(sc + 4 * kScEnd);
        Block wu = U;
#pragma unroll
        for (int a = 0; a < 2; a++)
#pragma unroll
            for (int e = 0; e < 4; e++) wu.t[a][e] *= wt.t[a][e];
        const Part<kParts> up = operand<kParts>(wu);
#pragma unroll
        for (int x = 0; x < KT; x++)
#pragma unroll
            for (int a = 0; a < 2; a++) {
#pragma unroll
                for (int e = 0; e < 4; e++) S[x].t[a][e] *= end;
                mm<kParts>(S[x].t[a], lane.column(at, x, a), up);
            }
        if (!SUM) {
            const Block sg = row_scalars(sc + 4 * kScG);
            const Part<kParts> op = operand<kParts>(U);
#pragma unroll
            for (int a = 0; a < 2; a++) {
#pragma unroll
                for (int e = 0; e < 4; e++) Y.t[a][e] *= sg.t[a][e];
            }
            lane.template matrix<kParts, kParts>(Y, at + L::p, op);
            leave(i, U, Y);
        }
    }
    if (!SUM)
#pragma unroll 1
        for (bool there = true; i < chunks; i++, there = false) {
            if (!there) {                                // the chunk that ended the loop above is there already
                meet_others();
                if (TRAIN)
#pragma unroll
                    for (int x = 0; x < KT; x++) state_keep(scratch, S[x], states, x, A.slices, slice);
            }
            Block U, Y;
            scan_rows<T, KT>(A, w, i, at0 + (i & 1) * L::size(A.slices), col, S, U, Y);
            leave(i, U, Y);
        }
    if (SUM) {
        if (values) state_write<KT>(S, A.starts + w.part * A.dk * A.dv, A.dk, A.dv, col);
        else {
            // the matrix, and for the backward its transpose, as delta_join takes them
            uint16_t *to = A.moves + w.part * A.move_size;
            const int g = l >> 4;
#pragma unroll
            for (int x = 0; x < KT; x++) {
                const Part<3> parts = operand<3>(S[x]);
#pragma unroll
                for (int n = 0; n < 3; n++) {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        *gp(to + move_at<KT>(32 * x + 8 * g + i, col) + 512 * n) = (uint16_t)(parts.p[n][i >> 1] >> 16 * (i & 1));
                    if (A.moves_back)
                        *gp(reinterpret_cast<u32x4_t *>(to + kMove<KT> + move_at<KT>(col, 32 * x + 8 * g) + 512 * n)) = parts.p[n];
                }
            }
        }
        return;
    }
    if (w.last) state_write<KT>(S, A.last + w.matrix * A.dk * A.dv, A.dk, A.dv, col);
}

// Walks backward, from the gradient of the last state.
template <typename T, int KT, bool SUM>
__global__ __launch_bounds__(576) void delta_back(DeltaArgs A)
{
    typedef WalkLds<T, KT, false> L;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const Walk w = walk_of(A);
    if (!w.any) return;
    const int slice = uniform((int)(threadIdx.x >> 6)), chunks = (w.rows + kCut - 1) / kCut;
    const uint32_t at0 = lds_address(lds);
    if (slice == A.slices) {
        bring_chunks<T, KT, false>(A, w, chunks, [=](int s) { return chunks - 1 - s; }, at0, A.dout, A.ds, A.dh);
        return;
    }
    const int l = lane_id(), r = l & 31, c = 16 * slice + 8 * (l >> 5), col = 16 * slice + (l & 15);
    const uint32_t scratch = at0 + 2 * L::size(A.slices) + slice * kScratch<T, true>;
    const Lane<T> lane;
    const uint32_t columns = lane.columns(slice);

    Block E[KT];
    state_read<KT>(E, SUM ? nullptr : A.cut ? A.starts + w.part * A.dk * A.dv : A.dlast ? A.dlast + w.matrix * A.dk * A.dv : nullptr,
                   A.dk, A.dv, col);
    const int64_t vstep = (int64_t)kCut * A.heads * A.dv, zstep = (int64_t)A.heads * A.slices * 2048,
                  sstep = (int64_t)A.heads * KT * A.slices * Lds<float>::kRows;
    T *dv = static_cast<T *>(A.dv_) + ((int64_t)(w.base + r) * A.heads + w.head) * A.dv + c + chunks * vstep;
    const int64_t number = (int64_t)w.tile0 * A.heads + w.head;
    char *z = static_cast<char *>(A.z) + (number * A.slices + slice) * 2048 + chunks * zstep;
    char *states = static_cast<char *>(A.e) + number * KT * A.slices * Lds<float>::kRows + chunks * sstep;
    auto leave = [&](int chunk, const Block &Z, const Block &dV) {
        rows_keep(scratch, Z, z);
        Turn<T> rows;
        rows.turn(scratch, dV);
        rows.write(dv, r < w.rows - chunk * kCut, c, A.dv, A.ovec);
    };
    int s = 0;
    for (; s < chunks; s++) {
        meet_others();
        const uint32_t at = at0 + (s & 1) * L::size(A.slices), sc = at + L::sc;
        dv -= vstep;
        z -= zstep;
        states -= sstep;
        Block X = zero_block();
#pragma unroll
        for (int x = 0; x < KT; x++) {
            const Part<kParts> ep = operand<kParts>(E[x]);
            if (!SUM) state_keep(scratch, E[x], states, x, A.slices, slice);
#pragma unroll
            for (int a = 0; a < 2; a++) mm<kParts>(X.t[a], lane.row(at, x, a), ep);
        }
        const Block wt = row_weights(sc);
        Block D = lane.block(at + L::v, columns);
        const Part<kIn<T>> dp = operand<kIn<T>>(D);
#pragma unroll
        for (int a = 0; a < 2; a++) {
#pragma unroll
            for (int e = 0; e < 4; e++) X.t[a][e] *= wt.t[a][e];
        }
        lane.template matrix_turned<kParts, kParts>(X, at + L::p, dp);
        const Part<kParts> xp = operand<kParts>(X);
        Block Z = X;
        lane.template matrix_turned<kParts, kParts>(Z, at + L::n, xp);
        if (!SUM && __builtin_expect(any_spoiled(Z), 0)) break;
        const Block bg = row_scalars(sc + 4 * kScBG), sg = row_scalars(sc + 4 * kScG);
        const float end = lds_read<float>(sc + 4 * kScEnd);
        Block gz = Z;
#pragma unroll
        for (int a = 0; a < 2; a++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                gz.t[a][e] *= -bg.t[a][e];
                D.t[a][e] *= sg.t[a][e];
            }
        const Part<kParts> zp = operand<kParts>(gz), op = operand<kParts>(D);
#pragma unroll
        for (int x = 0; x < KT; x++)
#pragma unroll
            for (int a = 0; a < 2; a++) {
#pragma unroll
                for (int e = 0; e < 4; e++) E[x].t[a][e] *= end;
                mm<kParts>(E[x].t[a], lane.column(at, x, a), zp);
                mm<kParts>(E[x].t[a], lane.column(at + L::q, x, a), op);
            }
        if (!SUM) {
            const Block b = row_scalars(sc + 4 * kScB);
            Block dV = Z;
#pragma unroll
            for (int a = 0; a < 2; a++)
#pragma unroll
                for (int e = 0; e < 4; e++) dV.t[a][e] *= b.t[a][e];
            leave(chunks - 1 - s, Z, dV);
        }
    }
    if (!SUM)
#pragma unroll 1
        for (bool there = true; s < chunks; s++, there = false) {
            if (!there) {
                meet_others();
                dv -= vstep;
                z -= zstep;
                states -= sstep;
#pragma unroll
                for (int x = 0; x < KT; x++) state_keep(scratch, E[x], states, x, A.slices, slice);
            }
            Block Z, dV;
            back_rows<T, KT>(A, w, chunks - 1 - s, at0 + (s & 1) * L::size(A.slices), col, E, Z, dV);
            leave(chunks - 1 - s, Z, dV);
        }
    if (SUM) {
        state_write<KT>(E, A.starts + w.part * A.dk * A.dv, A.dk, A.dv, col);
        return;
    }
    if (w.first && A.dstate) state_write<KT>(E, A.dstate + w.matrix * A.dk * A.dv, A.dk, A.dv, col);
}

// The states at the edges of a cut sample's segments, one after another: S' = move S + added
// (BACK: from the last, with the move transposed).  A wavefront has 16 columns of a sample's
// and head's state, four of them (one a SIMD) share a workgroup and a fifth that brings the
// moves, 32 of their columns at a time and up to kJoinAhead such steps ahead (three: 75 us for
// the below).  They come in the parts that the products take: cut into them by every wavefront
// again, they took most of the time.  64 segments of 64 x 128: 190 us then, 69 us so, a latency of
// 1.1 us a segment.  What a segment adds is replaced by the state that it begins with.
constexpr int kJoined = 4;
// steps on their way behind the one that is waited for (at most 63 loads are counted), and places
template <int KT>
constexpr int kJoinAhead = KT == 1 ? 6 : 10 / KT;
template <int KT>
constexpr int kJoinRing = kJoinAhead<KT> + 2;

template <int KT, bool BACK>
__global__ __launch_bounds__(64 * kJoined + 64) void delta_join(DeltaArgs A)
{
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    constexpr int pieces = 6 * KT, stage = pieces * 1024;
    const int sample = blockIdx.x / (uint32_t)A.heads, head = blockIdx.x - (uint32_t)sample * (uint32_t)A.heads;
    const int l = lane_id(), wave = uniform((int)(threadIdx.x >> 6)), slice = blockIdx.y * kJoined + wave, col = 16 * slice + (l & 15);
    const int base = uniform(seg_edge(A.off, A.samples, A.n, sample + 1));
    const int rows = max(uniform(seg_edge(A.off, A.samples, A.n, sample + 2)) - base, 0);
    const int parts = (rows + kSpan - 1) / kSpan, part0 = base / kSpan + sample + 1;
    const int64_t matrix = (int64_t)sample * A.heads + head;
    const uint32_t at0 = lds_address(lds);
    auto number = [&](int j) { return (int64_t)(part0 + (BACK ? parts - 1 - j : j)) * A.heads + head; };
    if (wave == kJoined) {
        const int steps = (parts - 1) * KT;
        int j = 0, x = 0, place = 0;                     // of the step that is asked for next
        auto bring = [&] {
            const i32x4_t rsrc = row_rsrc(A.moves + number(j) * A.move_size + (BACK ? kMove<KT> : 0) + x * (stage / 2));
            const uint32_t to = (uint32_t)uniform((int)(at0 + place * stage));
#pragma unroll
            for (int p = 0; p < pieces; p++) load_to_lds(rsrc, to + p * 1024, 16 * l, p * 1024);
            if (++x == KT) x = 0, j++;
            if (++place == kJoinRing<KT>) place = 0;
        };
        for (int s = 0; s < min(steps, kJoinAhead<KT> + 1); s++) bring();
        for (int s = 0; s < steps; s++) {
            // step s is there if only the ones behind it, asked for already, may be missing
            if (s + kJoinAhead<KT> < steps) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kJoinAhead<KT> * pieces) : "memory");
            else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            meet_others();                               // and everyone is done with step s - 1
            if (s + kJoinAhead<KT> + 1 < steps) bring();
        }
        return;
    }
    if (slice >= A.slices) return;
    const float *from = BACK ? A.dlast : A.state;
    // What is added is read two segments ahead, so that its wait is not one for the stores between.
    // Registers change roles instead of places: a copy would wait for what is on its way.
    Block S[KT], one[KT], two[KT], three[KT];
    state_read<KT>(S, from ? from + matrix * A.dk * A.dv : nullptr, A.dk, A.dv, col);
    if (parts) state_read<KT>(one, A.starts + number(0) * A.dk * A.dv, A.dk, A.dv, col);
    if (parts > 1) state_read<KT>(two, A.starts + number(1) * A.dk * A.dv, A.dk, A.dv, col);
    if (parts) state_write<KT>(S, A.starts + number(0) * A.dk * A.dv, A.dk, A.dv, col);
    int place = 0;
    auto step = [&](int j, const Block(&S)[KT], Block(&added)[KT], Block(&after)[KT]) {
        if (j + 1 >= parts) return false;
        if (j + 2 < parts) state_read<KT>(after, A.starts + number(j + 2) * A.dk * A.dv, A.dk, A.dv, col);
#pragma unroll
        for (int x = 0; x < KT; x++) {
            const Part<3> sp = operand<3>(S[x]);
            meet_others();
            const uint32_t at = at0 + place * stage;
            if (++place == kJoinRing<KT>) place = 0;
#pragma unroll
            for (int y = 0; y < KT; y++)
#pragma unroll
                for (int a = 0; a < 2; a++) mm<3>(added[y].t[a], staged<3>(at, 2 * y + a), sp);
        }
        state_write<KT>(added, A.starts + number(j + 1) * A.dk * A.dv, A.dk, A.dv, col);
        return true;
    };
    for (int j = 0;; j += 4)
        if (!step(j, S, one, three) || !step(j + 1, one, two, S) || !step(j + 2, two, three, one) || !step(j + 3, three, S, two)) break;
    if (parts) return;                                   // a sample without rows hands its state on
    float *to = BACK ? A.dstate : A.last;
    if (to) state_write<KT>(S, to + matrix * A.dk * A.dv, A.dk, A.dv, col);
}

// ----------------------------------------------------------------- gradients

// 32 rows x 16 elements of a state kept as an operand in memory
struct Kept {
    u32x4_t w[2];

    __device__ __forceinline__ void load(const char *at, int x)
    {
#pragma unroll
        for (int j = 0; j < 2; j++)
            w[j] = *gp(reinterpret_cast<const u32x4_t *>(at + x * Lds<float>::kRows + j * 1024) + lane_id());
    }
    __device__ __forceinline__ Part<3> operand() const
    {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] = __uint_as_float(w[j >> 2][j & 3]);
        return split8<3>(f);
    }
};

template <typename T, int KT>
struct GradLds {
    static constexpr int q = 2 * KT * Lds<T>::kRows, sc = 2 * q, with = sc + 1024, u = with + 6 * kParts * 1024;
    static __host__ __device__ int size(int slices) { return u + slices * (2 * 2048 + Lds<T>::kRows); }
};

// One chunk and key head: wavefront w makes columns 32 w .. of dq and dk.  What rows of K and Q
// are taken with, D, D^T and B + B^T, is made by a wavefront each and handed over in LDS; the
// first makes dgate and dbeta.  Bound by what it reads, half of it the two sides' states.
template <typename T, int KT>
__global__ __launch_bounds__(64 * KT, 2) void delta_grads(DeltaArgs A)
{
    typedef GradLds<T, KT> L;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    __shared__ float red[KT][3][32], cross[3][32], owns[32];
    const int tile = blockIdx.x, key = blockIdx.y;
    const int wave = uniform((int)(threadIdx.x >> 6)), l = lane_id(), c = l & 31, h = l >> 5;
    const SegTile s = seg_find<kCut>(A.off, A.n, nullptr, 0, A.samples, 1, tile);
    if (s.row0 >= s.rows) return;
    const int left = min(s.rows - s.row0, kCut);
    const int64_t row = (int64_t)s.base + s.row0;
    if (s.seg == 0 || s.seg == A.samples + 1) {          // rows of no sample
        const int g0 = key * A.group;
        for (int r = 0; r < left; r++) {
            for (int x = threadIdx.x; x < A.dk; x += 64 * KT) {
                const int64_t at = ((row + r) * A.key_heads + key) * A.dk + x;
                Row<T>::put1(static_cast<T *>(A.dq) + at, 0.f);
                Row<T>::put1(static_cast<T *>(A.dk_) + at, 0.f);
            }
            for (int x = threadIdx.x; x < A.group * A.dv; x += 64 * KT)
                Row<T>::put1(static_cast<T *>(A.dv_) + ((row + r) * A.heads + g0) * A.dv + x, 0.f);
            for (int x = threadIdx.x; x < A.group; x += 64 * KT) {
                Row<T>::put1(static_cast<T *>(A.dgate) + (row + r) * A.heads + g0 + x, 0.f);
                Row<T>::put1(static_cast<T *>(A.dbeta) + (row + r) * A.heads + g0 + x, 0.f);
            }
        }
        return;
    }
    const bool valid = c < left;
    const bool keep = valid && (!A.mask || *gp(A.mask + row + c));
    const uint32_t kept = (uint32_t)__ballot(keep);
    const uint32_t at = lds_address(lds);
    const uint32_t columns = Lds<T>::column();
    auto bring = [&](int head) {
        const int64_t number = (int64_t)tile * A.heads + head;
        const int n = A.slices;
        if (wave == 0) load_to_lds(row_rsrc(A.rec + number * A.rec_size), at + L::sc, 16 * l + (l < kScWalk / 4 ? Rec::sc : Rec::more - kScWalk * 4), 0);
        bring_flat(row_rsrc(static_cast<const char *>(A.u) + number * n * 2048), at + L::u, 2 * n, wave, KT);
        bring_flat(row_rsrc(static_cast<const char *>(A.z) + number * n * 2048), at + L::u + n * 2048, 2 * n, wave, KT);
        bring_rows<T>(row_rsrc(static_cast<const T *>(A.dout) + row * A.ds + head * A.dh), row_at<T>(kept, A.ds),
                      at + L::u + 2 * n * 2048, n, wave, KT);
    };
    bring_rows<T>(row_rsrc(static_cast<const T *>(A.k) + row * A.ks + key * A.kh), row_at<T>(kept, A.ks), at, 2 * KT, wave, KT);
    bring_rows<T>(row_rsrc(static_cast<const T *>(A.q) + row * A.qs + key * A.qh), row_at<T>(kept, A.qs), at + L::q, 2 * KT, wave, KT);
    bring(key * A.group);
    f32x16_t dq = zero16(), dk = zero16();               // transposed: a row a lane
    bool spoiled = false;
    for (int g = 0; g < A.group; g++) {
        const int head = key * A.group + g;
        if (g) {
            __syncthreads();                             // the head before is read
            bring(head);
        }
        const int64_t number = (int64_t)tile * A.heads + head, n = A.slices;
        const char *S0 = static_cast<const char *>(A.s0) + (number * KT + wave) * n * Lds<float>::kRows;
        const char *E0 = static_cast<const char *>(A.e) + (number * KT + wave) * n * Lds<float>::kRows;
        const uint32_t sc = at + L::sc, uat = at + L::u, zat = uat + n * 2048, oat = zat + n * 2048;
        meet();
        const float b = lds_read<float>(sc + 4 * (kScB + c)), bg = lds_read<float>(sc + 4 * (kScBG + c)),
                    sg = lds_read<float>(sc + 4 * (kScG + c)), wt = c == 31 ? 1.f : lds_read<float>(sc + 4 * (kScW + c)),
                    hi = lds_read<float>(sc + 4 * (kScHi + c)), lo = lds_read<float>(sc + 4 * (kScLo + c)),
                    end = lds_read<float>(sc + 4 * kScEnd);
        // lane x: what k_y (or q_y) is taken with, in register y; `across`: the lane's row or
        // column sum of H
#pragma unroll
        for (int what = 0; what < 3; what++) {
            if (what % KT != wave) continue;
            f32x16_t p = zero16(), p2 = zero16(), k = zero16(), f;
            for (int x = 0; x < n; x++) {
                const auto U = Lds<float>::rows(uat, x);
                if (what == 2) {
                    const auto Z = Lds<float>::rows(zat, x);
                    mm<kParts>(p, U, Z);                 // u_j.z_i, lane i
                    mm<kParts>(p2, Z, U);                // z_i.u_j, lane j
                } else {
                    const auto D = Lds<T>::rows(oat, x);
                    if (what == 0) mm<kParts>(p, U, D); // u_j.dO_i, lane i
                    else mm<kParts>(p, D, U);            // dO_i.u_j, lane j
                }
            }
#pragma unroll
            for (int x = 0; x < 2 * KT; x++) {
                const auto K = Lds<T>::rows(at, x);
                if (what == 2) mm<kIn<T>>(k, K, K);
                else {
                    const auto Q = Lds<T>::rows(at + L::q, x);
                    if (what == 0) mm<kIn<T>>(k, K, Q);
                    else mm<kIn<T>>(k, Q, K);
                }
            }
            float across = 0.f, own = 0.f;               // own: z.u of the row
#pragma unroll
            for (int g4 = 0; g4 < 4; g4++) {
                const int y0 = 8 * g4 + 4 * h;
                const f32x4_t yhi = lds_read<f32x4_t>(sc + 4 * (kScHi + y0)), ylo = lds_read<f32x4_t>(sc + 4 * (kScLo + y0)),
                              yb = lds_read<f32x4_t>(sc + 4 * (kScB + y0));
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int y = y0 + e, r = 4 * g4 + e;
                    const bool before = y < c, after = y > c;
                    const float dhi = hi - yhi[e], dlo = lo - ylo[e];
                    if (what == 0) {                     // D_xy
                        f[r] = !after ? A.scale * exp_of(dhi, dlo) * p[r] : 0.f;
                        across += before ? f[r] * k[r] : 0.f;
                    } else if (what == 1) {              // D_yx
                        f[r] = !before ? A.scale * exp_of(-dhi, -dlo) * p[r] : 0.f;
                        across -= after ? f[r] * k[r] : 0.f;
                    } else {                             // B_xy or B_yx
                        const float d = exp_of(before ? dhi : -dhi, before ? dlo : -dlo);
                        f[r] = before ? -b * d * p[r] : after ? -yb[e] * d * p2[r] : 0.f;
                        const float x = f[r] * k[r];
                        across += before ? x : -x;
                        if (y == c) own += p[r];
                    }
                }
            }
#pragma unroll
            for (int kc = 0; kc < 2; kc++) {
                const Part<kParts> o = operand<kParts>(f, kc);
#pragma unroll
                for (int i = 0; i < kParts; i++)
                    lds_write(at + L::with + ((what * 2 + kc) * kParts + i) * 1024 + 16 * l, o.p[i]);
            }
            across = both(across);
            if (h == 0) cross[what][c] = across;
            if (what == 2) {
                own = both(own);
                if (h == 0) owns[c] = own;
            }
        }
        __syncthreads();
        // the states' rows: 16 columns a step, the next step's on their way (all of them on their way from
        // the start: one wavefront a SIMD instead of two)
        Kept S[2], E[2];
        S[0].load(S0, 0);
        E[0].load(E0, 0);
#pragma unroll
        for (int kc = 0; kc < 2; kc++) {
            const auto kt = Lds<T>::turned(at, columns, wave, kc), qt = Lds<T>::turned(at + L::q, columns, wave, kc);
            mm<kParts>(dq, kt, staged<kParts>(at + L::with, kc));
            mm<kParts>(dk, kt, staged<kParts>(at + L::with, 4 + kc));
            mm<kParts>(dk, qt, staged<kParts>(at + L::with, 2 + kc));
        }
        // with the states: rows of S and E by rows of dO, Z and U, and the rows' own products of S and E
        f32x16_t t1 = zero16(), t2 = zero16(), t3 = zero16();
        float inner = 0.f;
#pragma unroll 1
        for (int x0 = 0; x0 < n; x0 += 2)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int x = x0 + i;
                if (x >= n) break;
                if (x + 1 < n) {
                    S[1 - i].load(S0, x + 1);
                    E[1 - i].load(E0, x + 1);
                }
                const auto s0 = S[i].operand();
                mm<kParts>(t1, s0, Lds<T>::rows(oat, x));
                mm<kParts>(t2, s0, Lds<float>::rows(zat, x));
                mm<kParts>(t3, E[i].operand(), Lds<float>::rows(uat, x));
#pragma unroll
                for (int j = 0; j < 8; j++) inner = fmaf(__uint_as_float(S[i].w[j >> 2][j & 3]), __uint_as_float(E[i].w[j >> 2][j & 3]), inner);
            }
        // the row's own elements 32 wave + kk(i, h), which meet its sums with the states
        float dots = 0.f, writes = 0.f;
#pragma unroll
        for (int g4 = 0; g4 < 4; g4++) {
            float fq[4], fk[4];
            Lds<T>::own(at + L::q, wave, g4, fq);
            Lds<T>::own(at, wave, g4, fk);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int i = 4 * g4 + e;
                const float x = sg * t1[i], y = -bg * t2[i], z = wt * t3[i];
                dq[i] += x;
                dk[i] += y + z;
                dots += fmaf(x, fq[e], y * fk[e]);
                writes = fmaf(z, fk[e], writes);
            }
        }
        dots = both(dots);
        writes = both(writes);
#pragma unroll
        for (int m = 1; m < 32; m *= 2) inner += __shfl_xor(inner, m, 64);
        inner = both(inner);
        if (h == 0) {
            red[wave][0][c] = dots;
            red[wave][1][c] = writes;
            red[wave][2][c] = inner;
        }
        __syncthreads();
        if (wave == 0) {
            float from = cross[0][c] + cross[1][c] + cross[2][c], into = 0.f, state = 0.f;
#pragma unroll
            for (int w = 0; w < KT; w++) {
                from += red[w][0][c];
                into += red[w][1][c];
                state += red[w][2][c];
            }
            float suffix = from, prefix = into;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const float x = __shfl_down(suffix, d, 32), y = __shfl_up(prefix, d, 32);
                if (c + d < 32) suffix += x;
                if (c >= d) prefix += y;
            }
            prefix = __shfl_up(prefix, 1, 32);           // of the rows before this one
            if (c == 0) prefix = 0.f;
            if (valid && h == 0) {
                float dg = 0.f, db = 0.f;
                if (keep) {
                    const float gate = Row<T>::get1(static_cast<const T *>(A.gate) + (row + c) * A.gs + head);
                    const float beta = Row<T>::get1(static_cast<const T *>(A.beta) + (row + c) * A.bs + head);
                    // a gate that forgets all has none, whatever the sums' rounding leaves
                    dg = expf(-gate) == INFINITY ? 0.f : (suffix + prefix + end * state) / (1.f + expf(gate));
                    db = owns[c] / (1.f + expf(beta));
                }
                spoiled = spoiled || fmaf(dg, 0.f, db * 0.f) != 0.f;
                Row<T>::put1(static_cast<T *>(A.dgate) + (row + c) * A.heads + head, dg);
                Row<T>::put1(static_cast<T *>(A.dbeta) + (row + c) * A.heads + head, db);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 16; i++) spoiled = spoiled || fmaf(dq[i], 0.f, dk[i] * 0.f) != 0.f;
    if (__builtin_expect(__syncthreads_or(spoiled), 0)) {
        // Something is not finite, and as products that reaches rows it has no part in: the chunk again by
        // the rule's own derivative, row by row from the last, the state before each made again.
        dq = dk = zero16();
        const int own = 32 * wave + c;                   // the lane's row of a state
        const bool there = own < A.dk;
        auto element = [&](uint32_t from, int r) {       // its element of row r of K or Q (zero where it is not there)
            const uint32_t in = (32 * (own >> 3 & 1) + r) * 16;
            if constexpr (sizeof(T) == 4) return lds_read<float>(from + (own >> 4) * 2048 + (own >> 2 & 1) * 1024 + in + (own & 3) * 4);
            else return bf16_lo((uint32_t)lds_read<uint16_t>(from + (own >> 4) * 1024 + in + (own & 7) * 2));
        };
        for (int g = 0; g < A.group; g++) {
            const int head = key * A.group + g, n = A.slices;
            const int64_t number = (int64_t)tile * A.heads + head;
            const uint32_t uat = at + L::u, zat = uat + n * 2048, oat = zat + n * 2048;
            __syncthreads();
            bring(head);
            meet();
            if (l < kCut) red[wave][0][l] = red[wave][1][l] = 0.f;
            if (wave == 0 && keep) cross[h][c] = logistic_at<T>(h ? A.beta : A.gate, (row + c) * (h ? A.bs : A.gs) + head);
            __syncthreads();
            // 16 columns at a time; rows of operands hold elements 8 h + 0 .. 7 of row r in lane 32 h + r
#pragma unroll 1
            for (int x = 0; x < n; x++) {
                float E[8], S[8], u[8], z[8], o[8];
                auto state = [&](const void *from, float (&f)[8]) {
                    Kept s;
                    s.load(static_cast<const char *>(from) + (number * KT + wave) * n * Lds<float>::kRows, x);
#pragma unroll
                    for (int e = 0; e < 8; e++) f[e] = there ? __uint_as_float(s.w[e >> 2][e & 3]) : 0.f;
                };
                auto fp32 = [&](uint32_t from, int r, float (&f)[8]) {
#pragma unroll
                    for (int e = 0; e < 8; e++) f[e] = lds_read<float>(from + x * 2048 + (e >> 2) * 1024 + (32 * h + r) * 16 + (e & 3) * 4);
                };
                state(A.e, E);
#pragma unroll 1
                for (int t = left - 1; t >= 0; t--) {
                    if (!(kept >> t & 1)) continue;
                    const float kt = element(at, t), qt = element(at + L::q, t), a = cross[0][t], b = cross[1][t];
                    state(A.s0, S);
#pragma unroll 1
                    for (int j = 0; j < t; j++) {
                        if (!(kept >> j & 1)) continue;
                        const float kj = element(at, j), aj = cross[0][j];
                        fp32(uat, j, u);
#pragma unroll
                        for (int e = 0; e < 8; e++) S[e] = fmaf(kj, u[e], aj * S[e]);
                    }
                    fp32(uat, t, u);
                    fp32(zat, t, z);
                    if constexpr (sizeof(T) == 4) fp32(oat, t, o);
                    else
#pragma unroll
                        for (int e = 0; e < 8; e++) o[e] = bf16_lo((uint32_t)lds_read<uint16_t>(oat + x * 1024 + (32 * h + t) * 16 + e * 2));
                    float sq = 0.f, sk = 0.f, da = 0.f, zu = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        if (!there || 16 * x + 8 * h + e >= A.dv) continue;
                        const float d = A.scale * o[e], bz = b * z[e], held = a * S[e];
                        const float f = fmaf(qt, d, E[e]), rest = fmaf(-kt, bz, f);
                        sq = fmaf(fmaf(kt, u[e], held), d, sq);
                        sk = fmaf(f, u[e], fmaf(-held, bz, sk));
                        da = fmaf(rest, S[e], da);
                        E[e] = a * rest;
                        zu = fmaf(z[e], u[e], zu);
                    }
                    sq = both(sq);
                    sk = both(sk);
                    zu = both(zu);
#pragma unroll
                    for (int m = 1; m < 32; m *= 2) da += __shfl_xor(da, m, 64);
                    da = both(da);
#pragma unroll
                    for (int i = 0; i < 16; i++) {       // rows of the state into registers, of the chunk into lanes
                        const float y = __shfl(sq, kk0(i) + 4 * h, 64), v = __shfl(sk, kk0(i) + 4 * h, 64);
                        dq[i] += c == t ? y : 0.f;
                        dk[i] += c == t ? v : 0.f;
                    }
                    if (l == 0) {                        // row 0 of a state is always there
                        red[wave][0][t] += da;
                        red[wave][1][t] += zu;
                    }
                }
            }
            __syncthreads();
            if (wave == 0 && h == 0 && keep) {
                float da = 0.f;
#pragma unroll
                for (int w = 0; w < KT; w++) da += red[w][0][c];
                const float gate = Row<T>::get1(static_cast<const T *>(A.gate) + (row + c) * A.gs + head);
                const float beta = Row<T>::get1(static_cast<const T *>(A.beta) + (row + c) * A.bs + head);
                const float a = 1.f / (1.f + expf(-gate));
                Row<T>::put1(static_cast<T *>(A.dgate) + (row + c) * A.heads + head, a * da / (1.f + expf(gate)));
                Row<T>::put1(static_cast<T *>(A.dbeta) + (row + c) * A.heads + head, red[0][1][c] / (1.f + expf(beta)));
            }
        }
    }
    if (!valid) return;
    const int64_t to = ((row + c) * A.key_heads + key) * A.dk;
#pragma unroll
    for (int g4 = 0; g4 < 4; g4++) {
        const int x0 = 32 * wave + 8 * g4 + 4 * h;
        float a[4], b[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            a[e] = dq[4 * g4 + e];
            b[e] = dk[4 * g4 + e];
        }
        if (A.vec) {
            if (x0 < A.dk) {
                Row<T>::put4(static_cast<T *>(A.dq) + to + x0, a);
                Row<T>::put4(static_cast<T *>(A.dk_) + to + x0, b);
            }
        } else {
            for (int e = 0; e < 4; e++)
                if (x0 + e < A.dk) {
                    Row<T>::put1(static_cast<T *>(A.dq) + to + x0 + e, a[e]);
                    Row<T>::put1(static_cast<T *>(A.dk_) + to + x0 + e, b[e]);
                }
        }
    }
}

// ------------------------------------------------------------- packed rows

// Rows of heads whose size is no multiple of 32, or that are not aligned to 16 bytes, as
// [n, heads, padded] with zeros behind each head.
template <typename T>
__global__ __launch_bounds__(256) void delta_pack(const T *x, int64_t xs, int64_t xh, T *y, int64_t n, int heads, int d,
                                                  int padded)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * heads * padded; i += (int64_t)gridDim.x * 256) {
        const int c = (int)(i % padded);
        const int64_t rh = i / padded;
        const int64_t r = rh / heads, h = rh % heads;
        *gp(y + i) = c < d ? *gp(x + r * xs + h * xh + c) : T(0);
    }
}

// ------------------------------------------------------------------ one step

constexpr int kStepThreads = 256;

// One row for one state [dk, dv] per workgroup.  Threads share the state as groups of rows
// times pieces of VEC columns, pieces a power of two; both products with the old state come
// from one pass, and o = scale (a S^T q + (q.k) u) needs no second one.
template <typename T, int VEC>
__global__ __launch_bounds__(kStepThreads) void delta_step(const T *q, int64_t qs, int64_t qh, const T *k, int64_t ks,
                                                           int64_t kh, const T *v, int64_t vs, int64_t vh, const T *gate,
                                                           int64_t gs, const T *beta, int64_t bs, float *state, T *o,
                                                           int heads, int group, int dk, int dv, int pieces, float scale)
{
    constexpr int kRows = 64 / VEC;              // most rows of a thread: 128 x 128 / (256 VEC)
    __shared__ float sq[kDeltaDim], sk[kDeltaDim];
    __shared__ float part[2][kStepThreads * VEC];
    __shared__ float su[kDeltaDim];
    const int64_t row = blockIdx.x / heads;
    const int head = blockIdx.x % heads, key = head / group;
    const int t = threadIdx.x;
    if (t < dk) sq[t] = Row<T>::get1(q + row * qs + key * qh + t);
    else if (t >= kDeltaDim && t - kDeltaDim < dk) sk[t - kDeltaDim] = Row<T>::get1(k + row * ks + key * kh + t - kDeltaDim);
    const int piece = t & (pieces - 1), r0 = t / pieces, step = kStepThreads / pieces, col = piece * VEC;
    float *S = state + ((row * heads + head) * dk) * dv;
    float s[kRows][VEC];
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        const int r = r0 + i * step;
#pragma unroll
        for (int e = 0; e < VEC; e++) s[i][e] = 0.f;
        if (r < dk && col < dv) {
            if (VEC == 4) {
                const f32x4_t x = *gp(reinterpret_cast<const f32x4_t *>(S + r * dv + col));
#pragma unroll
                for (int e = 0; e < VEC; e++) s[i][e] = x[e];
            } else s[i][0] = *gp(S + r * dv + col);
        }
    }
    const float g = Row<T>::get1(gate + row * gs + head), x = Row<T>::get1(beta + row * bs + head);
    const float a = 1.f / (1.f + expf(-g)), b = 1.f / (1.f + expf(-x));
    const float val = t < dv ? Row<T>::get1(v + row * vs + head * vh + t) : 0.f;
    __syncthreads();
    float ks_[VEC], qs_[VEC];
#pragma unroll
    for (int e = 0; e < VEC; e++) ks_[e] = qs_[e] = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        const int r = r0 + i * step;
        if (r < dk) {
            const float kr = sk[r], qr = sq[r];
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                s[i][e] *= a;
                ks_[e] = fmaf(kr, s[i][e], ks_[e]);
                qs_[e] = fmaf(qr, s[i][e], qs_[e]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; e++) {
        part[0][r0 * pieces * VEC + col + e] = ks_[e];
        part[1][r0 * pieces * VEC + col + e] = qs_[e];
    }
    __syncthreads();
    if (t < dv) {
        float x0 = 0.f, x1 = 0.f, qk = 0.f;
        for (int r = 0; r < step; r++) {
            x0 += part[0][r * pieces * VEC + t];
            x1 += part[1][r * pieces * VEC + t];
        }
        for (int r = 0; r < dk; r++) qk = fmaf(sq[r], sk[r], qk);
        const float u = b * (val - x0);
        su[t] = u;
        Row<T>::put1(o + (row * heads + head) * dv + t, scale * fmaf(qk, u, x1));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        const int r = r0 + i * step;
        if (r < dk && col < dv) {
            const float kr = sk[r];
            if (VEC == 4) {
                f32x4_t y;
#pragma unroll
                for (int e = 0; e < VEC; e++) y[e] = fmaf(kr, su[col + e], s[i][e]);
                *gp(reinterpret_cast<f32x4_t *>(S + r * dv + col)) = y;
            } else *gp(S + r * dv + col) = fmaf(kr, su[col], s[i][0]);
        }
    }
}

}  // namespace emb

using namespace emb;

namespace {

constexpr int64_t kDeltaStrideMost = int64_t(1) << 21;      // 32 rows of fp32 within a buffer's 2^31 bytes

size_t pad256(size_t x) { return (x + 255) & ~size_t(255); }

emb_status delta_check(const emb_delta *d)
{
    if (d->dtype != EMB_F32 && d->dtype != EMB_BF16) return fail(EMB_ERR_INVALID_ARG, "delta rule: unknown dtype");
    if (d->samples < 0 || d->n < 0) return fail(EMB_ERR_INVALID_ARG, "delta rule: samples and n must be >= 0");
    if (d->heads < 1 || d->key_heads < 1 || d->heads % d->key_heads)
        return fail(EMB_ERR_INVALID_ARG, "delta rule: heads must be a multiple of key_heads, both >= 1");
    if (d->dk < 1 || d->dv < 1) return fail(EMB_ERR_INVALID_ARG, "delta rule: dk and dv must be >= 1");
    if (d->dk > kDeltaDim || d->dv > kDeltaDim) return fail(EMB_ERR_UNSUPPORTED, "delta rule: dk and dv must be <= 128");
    if (d->heads > 65535 || d->heads * (int64_t)(d->dk > d->dv ? d->dk : d->dv) > kDeltaStrideMost)
        return fail(EMB_ERR_UNSUPPORTED, "delta rule: heads must be <= 65535, and heads x dk and x dv <= 2^21");
    if (!(d->scale >= -1e18f && d->scale <= 1e18f)) return fail(EMB_ERR_INVALID_ARG, "delta rule: scale must be finite");
    if (d->n > kRowsMost || d->samples > (1 << 24))
        return fail(EMB_ERR_UNSUPPORTED, "delta rule: n must be <= 2^31 - 65536 and samples <= 2^24");
    const int64_t all[] = {d->q_stride, d->q_head_stride, d->k_stride, d->k_head_stride, d->v_stride, d->v_head_stride,
                           d->gate_stride, d->beta_stride};
    for (int64_t s : all)
        if (s < 0) return fail(EMB_ERR_INVALID_ARG, "delta rule: strides must be >= 0");
    // the stride of a single row leads nowhere
    if (d->n > 1 && (d->q_stride > kDeltaStrideMost || d->k_stride > kDeltaStrideMost || d->v_stride > kDeltaStrideMost))
        return fail(EMB_ERR_UNSUPPORTED, "delta rule: row strides must be <= 2^21");
    return EMB_OK;
}

emb_status delta_pointers(const emb_delta *d)
{
    const size_t el = d->dtype == EMB_BF16 ? 2 : 4;
    if (!d->offsets || !aligned(d->offsets, 4)) return fail(EMB_ERR_INVALID_ARG, "delta rule: offsets must be given");
    if (d->n && (!d->q || !d->k || !d->v || !d->gate || !d->beta))
        return fail(EMB_ERR_INVALID_ARG, "delta rule: q, k, v, gate and beta must be given");
    for (const void *p : {d->q, d->k, d->v, d->gate, d->beta})
        if (!aligned(p, el)) return fail(EMB_ERR_INVALID_ARG, "delta rule: inputs must be aligned to their elements");
    if (!aligned(d->state, 4)) return fail(EMB_ERR_INVALID_ARG, "delta rule: state must be 4-byte aligned");
    return EMB_OK;
}

// rows of heads that the kernels read as they are: whole blocks of 32 elements, 16-byte aligned
bool rows_ready(const void *p, int64_t stride, int64_t head_stride, int dim, size_t el)
{
    return dim % 32 == 0 && aligned(p, 16) && stride * el % 16 == 0 && head_stride * el % 16 == 0;
}

struct DeltaPlan {
    size_t el;
    int kt, slices;
    int64_t tiles;
    bool cut;
    size_t rec, move;                        // bytes of a record, of a segment's matrix
    size_t recs, states, us, moves, starts;  // bytes of all of them
    int ranks;                               // workgroups that order the samples
    size_t order;
    size_t q, k, v;                          // bytes of packed rows, 0 where they are read in place
    size_t saved, forward, backward;
};

// Samples are cut into segments where there are too few of them, times the heads, to fill the
// chip.  A cut walk is walked twice and its segments are joined one after another.  Uncut and
// cut, forward / with the backward, in us, 4 heads of dk x dv:
//   walks x rows      4 x 2048         4 x 16384        32 x 2048       64 x 2048        64 x 4096        128 x 4096
//   bf16 64 x 64      101, 257         696, 1784        106, 297        112, 350         207, 674         246, 930
//                     95, 231          119, 305         103, 275        117, 344         171, 602         281, 1061
//   bf16 128 x 128    183, 495         1349, 3694       189, 601        205, 777         394, 1536        464, 2187
//                     171, 443         227, 630         186, 544        238, 787         415, 1443        693, 2514
//   fp32 64 x 64      194, 440         1435, 3231       202, 511        210, 598         407, 1176        451, 1543
//                     173, 405         200, 509         182, 482        217, 607         335, 1049        524, 1778
//   fp32 128 x 128    462, 1019        3577, 7939       475, 1202       491, 1415        972, 2801        1066, 3668
//                     408, 937         467, 1213        425, 1125       595, 1510        1039, 2815       1671, 4713
// 4 x 1024 rows take half as long uncut in all of them.
bool delta_cut(const emb_delta *d)
{
    const int64_t walks = (int64_t)d->samples * d->heads;
    return d->samples && walks <= 64 && d->n / d->samples >= (walks <= 32 ? 2 : 4) * kSpan;
}

DeltaPlan delta_plan(const emb_delta *d, bool train)
{
    DeltaPlan p{};
    p.el = d->dtype == EMB_BF16 ? 2 : 4;
    p.kt = (d->dk + 31) / 32;
    p.slices = (d->dv + 15) / 16;
    p.tiles = seg_tiles(d->n, d->samples, 1, kCut);
    p.cut = delta_cut(d);
    p.rec = Rec::size;
    p.recs = (size_t)p.tiles * d->heads * p.rec;
    p.us = (size_t)p.tiles * d->heads * p.slices * 2048;
    p.states = (size_t)p.tiles * d->heads * p.slices * p.kt * 2048;
    if (p.cut) {
        const size_t segments = (size_t)seg_tiles(d->n, d->samples, 1, kSpan) * d->heads;
        p.move = (size_t)p.kt * p.kt * 6144 * (train ? 2 : 1);
        p.moves = segments * p.move;
        p.starts = pad256(segments * d->dk * d->dv * 4);
    }
    // Where there are more walks than CUs.  Forward / with the backward in us, the samples' own order
    // and the longest first, bf16 heads of 64: 256 x 200..2000 rows, 4 heads: 473, 1906 and 420, 1813; 300 x
    // 10..3000, 1 head: 225, 899 and 193, 765; 1024 x 50..800, 4 heads: 580, 2697 and 564, 2663;
    // 256 x 1000: the same.  More and shorter samples are even enough by themselves (4000 x 20..200,
    // 4 heads: 632, 3018 and 646, 3082).
    if (!p.cut && (int64_t)d->samples * d->heads > 256 && d->samples <= kRanked && d->n / d->samples >= 64) {
        p.ranks = (d->samples + 63) / 64;
        p.order = (size_t)p.ranks * 256;
    }
    const size_t keys = pad256((size_t)d->n * d->key_heads * p.kt * 32 * p.el);
    p.q = rows_ready(d->q, d->q_stride, d->q_head_stride, d->dk, p.el) ? 0 : keys;
    p.k = rows_ready(d->k, d->k_stride, d->k_head_stride, d->dk, p.el) ? 0 : keys;
    const size_t values = pad256((size_t)d->n * d->heads * ((d->dv + 31) / 32 * 32) * p.el);
    p.v = rows_ready(d->v, d->v_stride, d->v_head_stride, d->dv, p.el) ? 0 : values;
    p.saved = p.order + p.recs + p.states + p.us + p.moves;
    p.forward = (train ? 0 : p.order + p.recs + p.moves) + p.starts + p.q + p.k + p.v;
    p.backward = p.states + p.us + p.starts + p.q + p.k + values;        // how dout lies is not known here
    return p;
}

emb_status delta_launched()
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(EMB_ERR_HIP, std::string("delta rule launch: ") + hipGetErrorString(e));
    return EMB_OK;
}

// rows as the kernels read them: in place, or packed into *ws, which moves on
constexpr int64_t kPackMost = int64_t(1) << 22;          // workgroups: below a launch's 2^32 threads
void delta_rows(const emb_delta *d, size_t packed, const void *&x, int64_t &xs, int64_t &xh, int heads, int dim, char *&ws,
                hipStream_t st)
{
    if (!packed) return;
    const int padded = (dim + 31) / 32 * 32;
    int64_t blocks = (d->n * heads * padded + 255) / 256;
    if (blocks > kPackMost) blocks = kPackMost;
    if (blocks && d->dtype == EMB_BF16)
        hipLaunchKernelGGL((delta_pack<uint16_t>), dim3((unsigned)blocks), dim3(256), 0, st, static_cast<const uint16_t *>(x),
                           xs, xh, reinterpret_cast<uint16_t *>(ws), d->n, heads, dim, padded);
    else if (blocks)
        hipLaunchKernelGGL((delta_pack<float>), dim3((unsigned)blocks), dim3(256), 0, st, static_cast<const float *>(x), xs,
                           xh, reinterpret_cast<float *>(ws), d->n, heads, dim, padded);
    x = ws;
    xh = padded;
    xs = (int64_t)padded * heads;
    ws += packed;
}

DeltaArgs delta_args(const emb_delta *d, const DeltaPlan &p)
{
    DeltaArgs A{};
    A.q = d->q;
    A.k = d->k;
    A.v = d->v;
    A.gate = d->gate;
    A.beta = d->beta;
    A.qs = d->q_stride;
    A.qh = d->q_head_stride;
    A.ks = d->k_stride;
    A.kh = d->k_head_stride;
    A.vs = d->v_stride;
    A.vh = d->v_head_stride;
    A.gs = d->gate_stride;
    A.bs = d->beta_stride;
    A.off = d->offsets;
    A.mask = d->mask;
    A.state = d->state;
    A.n = (int32_t)d->n;
    A.samples = d->samples;
    A.key_heads = d->key_heads;
    A.heads = d->heads;
    A.group = d->heads / d->key_heads;
    A.dk = d->dk;
    A.dv = d->dv;
    A.slices = p.slices;
    A.scale = d->scale;
    A.rec_size = (int64_t)p.rec;
    A.cut = p.cut;
    A.move_size = (int64_t)p.move / 2;
    return A;
}

// the samples' order, records, states, U and the segments' matrices in the buffer that the forward
// leaves for the backward
void delta_saved(const DeltaPlan &p, DeltaArgs &A, char *saved)
{
    A.order = p.order ? reinterpret_cast<int32_t *>(saved) : nullptr;
    A.rec = saved + p.order;
    A.s0 = A.rec + p.recs;
    A.u = A.rec + p.recs + p.states;
    A.moves = reinterpret_cast<uint16_t *>(A.rec + p.recs + p.states + p.us);
}

int64_t delta_walks(const emb_delta *d, const DeltaPlan &p)
{
    return (p.cut ? seg_tiles(d->n, d->samples, 1, kSpan) : d->samples) * d->heads;
}

emb_status delta_sizes(const emb_delta *d, const DeltaPlan &p, bool train)
{
    // a launch's threads in one dimension are counted in 32 bits
    const int64_t most = (int64_t(1) << 32) - 1, tiles = p.tiles + p.ranks;
    const int slices = p.cut && p.slices < 2 * p.kt ? 2 * p.kt : p.slices;
    if (tiles > most / (64 * (train ? p.kt : 1)) || delta_walks(d, p) > most / (64 * slices + 64))
        return fail(EMB_ERR_UNSUPPORTED, "delta rule: too many rows, or samples x heads, for one launch");
    return EMB_OK;
}

template <typename F>
void delta_launch(F kernel, dim3 grid, int threads, size_t lds, const DeltaArgs &A, hipStream_t st)
{
    // more LDS than every chip has is asked for by name
    if (lds > 65536)
        (void)hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    hipLaunchKernelGGL(kernel, grid, dim3((unsigned)threads), lds, st, A);
}

template <typename T, int KT>
void delta_forward_launch(const DeltaArgs &A, int64_t tiles, int64_t walks, bool train, hipStream_t st)
{
    const dim3 walk((unsigned)walks);
    const int join = kJoinRing<KT> * KT * 6144;
    const dim3 joins((unsigned)(A.samples * A.heads), (unsigned)((A.slices + kJoined - 1) / kJoined));
    delta_launch(delta_prepare<T, KT>, dim3((unsigned)(A.ranks + tiles), (unsigned)A.heads), 64, 0, A, st);
    if (!walks) return;
    if (A.cut) {
        // wavefronts enough for either kind
        const int most = A.slices > 2 * KT ? A.slices : 2 * KT;
        delta_launch(delta_scan<T, KT, false, true>, dim3((unsigned)walks, 2), 64 * most + 64, 2 * WalkLds<T, KT, true>::size(A.slices),
                     A, st);
        delta_launch(delta_join<KT, false>, joins, 64 * kJoined + 64, join, A, st);
    }
    const int stages = 2 * WalkLds<T, KT, false>::size(A.slices), threads = 64 * A.slices + 64;
    if (train) delta_launch(delta_scan<T, KT, true, false>, walk, threads, stages + A.slices * kScratch<T, true>, A, st);
    else delta_launch(delta_scan<T, KT, false, false>, walk, threads, stages + A.slices * kScratch<T, false>, A, st);
}

template <typename T, int KT>
void delta_backward_launch(const DeltaArgs &A, int64_t tiles, int64_t walks, bool, hipStream_t st)
{
    const dim3 walk((unsigned)walks);
    const int lds = 2 * WalkLds<T, KT, false>::size(A.slices), join = kJoinRing<KT> * KT * 6144;
    const dim3 joins((unsigned)(A.samples * A.heads), (unsigned)((A.slices + kJoined - 1) / kJoined));
    if (walks && A.cut) {
        delta_launch(delta_back<T, KT, true>, walk, 64 * A.slices + 64, lds, A, st);
        delta_launch(delta_join<KT, true>, joins, 64 * kJoined + 64, join, A, st);
    }
    if (walks) delta_launch(delta_back<T, KT, false>, walk, 64 * A.slices + 64, lds + A.slices * kScratch<T, true>, A, st);
    delta_launch(delta_grads<T, KT>, dim3((unsigned)tiles, (unsigned)A.key_heads), 64 * KT, GradLds<T, KT>::size(A.slices), A, st);
}

#define EMB_DELTA_SIZES(NAME, T)                             \
    (p.kt == 1   ? NAME<T, 1>(A, p.tiles, walks, train, st)  \
     : p.kt == 2 ? NAME<T, 2>(A, p.tiles, walks, train, st)  \
     : p.kt == 3 ? NAME<T, 3>(A, p.tiles, walks, train, st)  \
                 : NAME<T, 4>(A, p.tiles, walks, train, st))

bool rows16(const void *x, int dim, size_t el) { return dim * el % 16 == 0 && aligned(x, 16); }

}  // namespace

extern "C" emb_status emb_delta_query(const emb_delta *d, int32_t training, size_t *saved_bytes, size_t *forward_bytes,
                                      size_t *backward_bytes)
{
    if (!d) return fail(EMB_ERR_INVALID_ARG, "delta rule descriptor is NULL");
    emb_status s = delta_check(d);
    if (s != EMB_OK) return s;
    if (!saved_bytes || !forward_bytes || !backward_bytes)
        return fail(EMB_ERR_INVALID_ARG, "delta rule: output pointers must be given");
    const DeltaPlan p = delta_plan(d, training != 0);
    s = delta_sizes(d, p, training != 0);
    if (s != EMB_OK) return s;
    *saved_bytes = training ? p.saved : 0;
    *forward_bytes = p.forward;
    *backward_bytes = training ? p.backward : 0;
    return EMB_OK;
}

extern "C" emb_status emb_delta_forward(const emb_delta *d, void *o, float *last, void *saved, void *workspace,
                                        size_t workspace_bytes, void *stream)
{
    if (!d) return fail(EMB_ERR_INVALID_ARG, "delta rule descriptor is NULL");
    emb_status s = delta_check(d);
    if (s == EMB_OK) s = delta_pointers(d);
    if (s != EMB_OK) return s;
    const bool train = saved != nullptr;
    const DeltaPlan p = delta_plan(d, train);
    if ((d->n && !o) || (d->samples && !last) || !aligned(o, p.el) || !aligned(last, 4) || !aligned(saved, 256))
        return fail(EMB_ERR_INVALID_ARG, "delta rule: o and last must be given and aligned, saved to 256 bytes");
    if (workspace_bytes < p.forward || (p.forward && (!workspace || !aligned(workspace, 256))))
        return fail(EMB_ERR_WORKSPACE, "delta rule: the workspace is smaller than the query returned, or not 256-byte aligned");
    s = delta_sizes(d, p, train);
    if (s != EMB_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    DeltaArgs A = delta_args(d, p);
    A.o = o;
    A.last = last;
    A.ovec = rows16(o, d->dv, p.el);
    A.moves_back = train;
    A.ranks = p.ranks;
    char *ws = static_cast<char *>(workspace);
    if (train) delta_saved(p, A, static_cast<char *>(saved));
    else {
        A.order = p.order ? reinterpret_cast<int32_t *>(ws) : nullptr;
        A.rec = ws + p.order;
        A.moves = reinterpret_cast<uint16_t *>(A.rec + p.recs);
        ws += p.order + p.recs + p.moves;
    }
    A.starts = reinterpret_cast<float *>(ws);
    ws += p.starts;
    delta_rows(d, p.q, A.q, A.qs, A.qh, d->key_heads, d->dk, ws, st);
    delta_rows(d, p.k, A.k, A.ks, A.kh, d->key_heads, d->dk, ws, st);
    delta_rows(d, p.v, A.v, A.vs, A.vh, d->heads, d->dv, ws, st);
    const int64_t walks = delta_walks(d, p);
    if (d->dtype == EMB_BF16) EMB_DELTA_SIZES(delta_forward_launch, uint16_t);
    else EMB_DELTA_SIZES(delta_forward_launch, float);
    return delta_launched();
}

extern "C" emb_status emb_delta_backward(const emb_delta *d, const void *saved, const void *dout, int64_t dout_stride,
                                         int64_t dout_head_stride, const float *dlast, void *dq, void *dk, void *dv,
                                         void *dgate, void *dbeta, float *dstate, void *workspace,
                                         size_t workspace_bytes, void *stream)
{
    if (!d) return fail(EMB_ERR_INVALID_ARG, "delta rule descriptor is NULL");
    emb_status s = delta_check(d);
    if (s == EMB_OK) s = delta_pointers(d);
    if (s != EMB_OK) return s;
    const bool train = true;
    const DeltaPlan p = delta_plan(d, train);
    if (!saved || !aligned(saved, 256)) return fail(EMB_ERR_INVALID_ARG, "delta rule: saved must be given, 256-byte aligned");
    if (d->n && (!dout || !dq || !dk || !dv || !dgate || !dbeta))
        return fail(EMB_ERR_INVALID_ARG, "delta rule: dout, dq, dk, dv, dgate and dbeta must be given");
    for (const void *x : {dout, (const void *)dq, (const void *)dk, (const void *)dv, (const void *)dgate,
                          (const void *)dbeta})
        if (!aligned(x, p.el)) return fail(EMB_ERR_INVALID_ARG, "delta rule: buffers must be aligned to their elements");
    if (!aligned(dlast, 4) || !aligned(dstate, 4))
        return fail(EMB_ERR_INVALID_ARG, "delta rule: buffers must be aligned to their elements");
    if (dout_stride < 0 || dout_head_stride < 0) return fail(EMB_ERR_INVALID_ARG, "delta rule: strides must be >= 0");
    if (d->n > 1 && dout_stride > kDeltaStrideMost) return fail(EMB_ERR_UNSUPPORTED, "delta rule: row strides must be <= 2^21");
    if (workspace_bytes < p.backward || (p.backward && (!workspace || !aligned(workspace, 256))))
        return fail(EMB_ERR_WORKSPACE, "delta rule: the workspace is smaller than the query returned, or not 256-byte aligned");
    s = delta_sizes(d, p, train);
    if (s != EMB_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    DeltaArgs A = delta_args(d, p);
    delta_saved(p, A, const_cast<char *>(static_cast<const char *>(saved)));
    char *ws = static_cast<char *>(workspace);
    A.e = ws;
    A.z = ws + p.states;
    A.starts = reinterpret_cast<float *>(ws + p.states + p.us);
    ws += p.states + p.us + p.starts;
    A.dout = dout;
    A.ds = dout_stride;
    A.dh = dout_head_stride;
    A.dlast = dlast;
    A.dq = dq;
    A.dk_ = dk;
    A.dv_ = dv;
    A.dgate = dgate;
    A.dbeta = dbeta;
    A.dstate = dstate;
    A.vec = d->dk % 4 == 0 && aligned(dq, 4 * p.el) && aligned(dk, 4 * p.el);
    A.ovec = rows16(dv, d->dv, p.el);
    delta_rows(d, p.q, A.q, A.qs, A.qh, d->key_heads, d->dk, ws, st);
    delta_rows(d, p.k, A.k, A.ks, A.kh, d->key_heads, d->dk, ws, st);
    const size_t values = rows_ready(dout, dout_stride, dout_head_stride, d->dv, p.el)
                              ? 0 : pad256((size_t)d->n * d->heads * ((d->dv + 31) / 32 * 32) * p.el);
    delta_rows(d, values, A.dout, A.ds, A.dh, d->heads, d->dv, ws, st);
    const int64_t walks = delta_walks(d, p);
    if (d->dtype == EMB_BF16) EMB_DELTA_SIZES(delta_backward_launch, uint16_t);
    else EMB_DELTA_SIZES(delta_backward_launch, float);
    return delta_launched();
}

extern "C" emb_status emb_delta_step(const emb_delta *d, float *state, void *o, void *stream)
{
    if (!d) return fail(EMB_ERR_INVALID_ARG, "delta rule descriptor is NULL");
    const emb_status s = delta_check(d);
    if (s != EMB_OK) return s;
    if (d->n == 0) return EMB_OK;
    const size_t el = d->dtype == EMB_BF16 ? 2 : 4;
    if (!d->q || !d->k || !d->v || !d->gate || !d->beta || !state || !o)
        return fail(EMB_ERR_INVALID_ARG, "delta rule step: q, k, v, gate, beta, state and o must be given");
    for (const void *p : {d->q, d->k, d->v, d->gate, d->beta, (const void *)o})
        if (!aligned(p, el)) return fail(EMB_ERR_INVALID_ARG, "delta rule step: buffers must be aligned to their elements");
    if (!aligned(state, 4)) return fail(EMB_ERR_INVALID_ARG, "delta rule step: state must be 4-byte aligned");
    if (d->n * d->heads > ((int64_t(1) << 32) - 1) / kStepThreads)
        return fail(EMB_ERR_UNSUPPORTED, "delta rule step: more than 2^24 - 1 states of one head");
    const bool four = d->dv % 4 == 0 && aligned(state, 16);
    int pieces = 1;
    while (pieces * (four ? 4 : 1) < d->dv) pieces *= 2;
    const dim3 grid((unsigned)(d->n * d->heads)), block(kStepThreads);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int group = d->heads / d->key_heads;
#define EMB_DELTA_STEP(T, VEC)                                                                                        \
    hipLaunchKernelGGL((delta_step<T, VEC>), grid, block, 0, st, static_cast<const T *>(d->q), d->q_stride,            \
                       d->q_head_stride, static_cast<const T *>(d->k), d->k_stride, d->k_head_stride,                  \
                       static_cast<const T *>(d->v), d->v_stride, d->v_head_stride, static_cast<const T *>(d->gate),   \
                       d->gate_stride, static_cast<const T *>(d->beta), d->beta_stride, state, static_cast<T *>(o),    \
                       d->heads, group, d->dk, d->dv, pieces, d->scale)
    if (d->dtype == EMB_BF16) {
        if (four) EMB_DELTA_STEP(uint16_t, 4);
        else EMB_DELTA_STEP(uint16_t, 1);
    } else {
        if (four) EMB_DELTA_STEP(float, 4);
        else EMB_DELTA_STEP(float, 1);
    }
#undef EMB_DELTA_STEP
    return delta_launched();
}
