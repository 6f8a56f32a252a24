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
// take 32 columns of the state per wavefront, which never meet one another.
//
// All products run on the matrix cores in 32 x 32 blocks (lane & 31 a column, register i of
// half h = lane >> 5 the row kk(i, h) = 8 (i >> 2) + 4 h + (i & 3)), which is also how the
// next product takes its second operand if its contraction runs in that order.  The state
// is fp32.  What enters a product is cut into bf16 parts, the first rounded from the value,
// the next from what is left of it: inputs in bf16 are one part, fp32 ones three (24 bits);
// the state and what makes it (N, U, Z, P^T) are three, so that the states that come out
// are fp32's; what only bf16 outputs are made of is two (16 bits), and the states, U and Z
// that the gradients read are kept as one.  Products of parts whose bits lie below the last
// part's are left out.
#include <string>

#include "sequence.h"

namespace emb {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kCut = 32;                 // rows of a chunk
constexpr int kDeltaDim = 128;           // largest head size
constexpr uint32_t kOut = 0x80000000u;   // an offset past every buffer: reads zero, writes nothing
// the scalars of a chunk and head, in floats
constexpr int kScB = 0, kScBG = 32, kScG = 64, kScW = 96, kScHi = 128, kScLo = 160, kScEnd = 192, kScKept = 193,
              kScalars = 256;

struct DeltaArgs {
    const void *q, *k, *v, *gate, *beta;            // rows and heads any stride apart (elements)
    int64_t qs, qh, ks, kh, vs, vh, gs, bs;
    const int32_t *off;
    const uint8_t *mask;
    const float *state;
    int32_t n, samples, key_heads, heads, group, dk, dv, slices;
    float scale;
    char *rec;                 // records of (tile, head): N, P, scalars (and N^T, P^T)
    char *recT;                // records of (tile, key head): K^T (and Q^T)
    int64_t rec_size, recT_size;
    void *s0, *u;              // saved for the backward: states [tile, head, dkp, dvp], U [n, heads, dvp]
    void *o;
    float *last;
    const void *dout;
    int64_t ds, dh;            // strides of dout
    const void *dop;           // dout as [n, heads, dvp], possibly itself
    int64_t dps, dph;
    const float *dlast;
    void *e, *z;               // E as s0, Z as u
    void *dq, *dk_, *dv_, *dgate, *dbeta;
    float *dstate;
    int32_t vec;               // dq and dk rows move in pieces of 4
};

// parts of the inputs, of what makes the states, and of what makes outputs alone
template <typename T>
struct Prec;
template <>
struct Prec<uint16_t> {
    static constexpr int IN = 1, ST = 3, OUT = 2;
};
template <>
struct Prec<float> {
    static constexpr int IN = 3, ST = 3, OUT = 3;
};

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
__device__ __forceinline__ u32x2_t buf8(__amdgpu_buffer_rsrc_t r, uint32_t at)
{
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, (int)at, 0, 0));
}

template <typename T>
struct Row;
// Rows in memory as operands, a row a lane: `at` is the byte offset of the lane's row (kOut for
// a row that reads as zero); natural(): elements 16 b + 8 h + 0 .. 7, turned(): elements
// 16 b + 8 (e >> 2) + 4 h + (e & 3), the order of a block's registers.
template <>
struct Row<uint16_t> {
    typedef Part<1> Op;
    static __device__ __forceinline__ Op natural(__amdgpu_buffer_rsrc_t r, uint32_t at, int h, int b)
    {
        return Op{{buf16(r, at + 32 * b + 16 * h)}};
    }
    static __device__ __forceinline__ Op turned(__amdgpu_buffer_rsrc_t r, uint32_t at, int h, int b)
    {
        const u32x2_t x = buf8(r, at + 32 * b + 8 * h), y = buf8(r, at + 32 * b + 16 + 8 * h);
        return Op{{u32x4_t{x[0], x[1], y[0], y[1]}}};
    }
    // the same as numbers
    static __device__ __forceinline__ void floats(__amdgpu_buffer_rsrc_t r, uint32_t at, int h, int b, float *f)
    {
        const Op o = turned(r, at, h, b);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            f[2 * j] = bf16_lo(o.p[0][j]);
            f[2 * j + 1] = bf16_hi(o.p[0][j]);
        }
    }
    static __device__ __forceinline__ float one(__amdgpu_buffer_rsrc_t r, uint32_t at)
    {
        return bf16_lo((uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)at, 0, 0));
    }
    static __device__ __forceinline__ void put(__amdgpu_buffer_rsrc_t r, uint32_t at, float v)
    {
        __builtin_amdgcn_raw_buffer_store_b16((short)bf16_rne(v), r, (int)at, 0, 0);
    }
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
    static __device__ __forceinline__ void read(__amdgpu_buffer_rsrc_t r, uint32_t x, uint32_t y, float *f)
    {
        const u32x4_t a = buf16(r, x), b = buf16(r, y);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            f[j] = __uint_as_float(a[j]);
            f[4 + j] = __uint_as_float(b[j]);
        }
    }
    static __device__ __forceinline__ Op natural(__amdgpu_buffer_rsrc_t r, uint32_t at, int h, int b)
    {
        float f[8];
        read(r, at + 64 * b + 32 * h, at + 64 * b + 32 * h + 16, f);
        return split8<3>(f);
    }
    static __device__ __forceinline__ void floats(__amdgpu_buffer_rsrc_t r, uint32_t at, int h, int b, float *f)
    {
        read(r, at + 64 * b + 16 * h, at + 64 * b + 32 + 16 * h, f);
    }
    static __device__ __forceinline__ Op turned(__amdgpu_buffer_rsrc_t r, uint32_t at, int h, int b)
    {
        float f[8];
        floats(r, at, h, b, f);
        return split8<3>(f);
    }
    static __device__ __forceinline__ float one(__amdgpu_buffer_rsrc_t r, uint32_t at)
    {
        return __int_as_float((int)__builtin_amdgcn_raw_buffer_load_b32(r, (int)at, 0, 0));
    }
    static __device__ __forceinline__ void put(__amdgpu_buffer_rsrc_t r, uint32_t at, float v)
    {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(v), r, (int)at, 0, 0);
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

// Operands that lie in memory as the lanes take them: 64 x 16 bytes a part.
template <int N>
__device__ __forceinline__ Part<N> load_frag(const char *at, int index)
{
    Part<N> r;
#pragma unroll
    for (int i = 0; i < N; i++)
        r.p[i] = *gp(reinterpret_cast<const u32x4_t *>(at) + (index * N + i) * 64 + lane_id());
    return r;
}
template <int N>
__device__ __forceinline__ void store_frag(char *at, int index, const Part<N> &f)
{
#pragma unroll
    for (int i = 0; i < N; i++)
        *gp(reinterpret_cast<u32x4_t *>(at) + (index * N + i) * 64 + lane_id()) = f.p[i];
}

// Where the pieces of a record lie: N, N^T and P^T of ST parts, P (which the state never
// meets) of OUT, the scalars.
template <typename T>
struct Rec {
    static constexpr int kN = 2 * Prec<T>::ST * 1024, kP = 2 * Prec<T>::OUT * 1024;
    static constexpr int n = 0, p = kN, sc = kN + kP, nt = sc + kScalars * 4, pt = nt + kN;
    static constexpr int small = nt, whole = pt + kN;
};

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

template <typename T, int KT, bool TRAIN>
__global__ __launch_bounds__(64) void delta_prepare(DeltaArgs A)
{
    constexpr int IN = Prec<T>::IN, ST = Prec<T>::ST, OUT = Prec<T>::OUT;
    constexpr int kPitch = 36;
    __shared__ __attribute__((aligned(16))) float lds[32 * kPitch];
    __shared__ __attribute__((aligned(16))) float sc[kScalars];
    const int tile = blockIdx.x, head = blockIdx.y, key = head / A.group;
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
        sc[kScW + c] = W;
        sc[kScHi + c] = hi;
        sc[kScLo + c] = lo;
        if (c == 31) sc[kScEnd] = G;
        if (c == 30) sc[kScKept] = __uint_as_float(kept);
    }
    wave_sync();
    char *rec = A.rec + ((int64_t)tile * A.heads + head) * A.rec_size;
    *gp(reinterpret_cast<f32x4_t *>(rec + Rec<T>::sc) + l) = *reinterpret_cast<const f32x4_t *>(sc + 4 * l);

    const auto qb = buffer<T>(A.q, row * A.qs + key * A.qh), kb = buffer<T>(A.k, row * A.ks + key * A.kh);
    const uint32_t qat = keep ? (uint32_t)(c * A.qs * sizeof(T)) : kOut;
    const uint32_t kat = keep ? (uint32_t)(c * A.ks * sizeof(T)) : kOut;
    f32x16_t kk = zero16(), kq = zero16(), qk = zero16();      // a lane's row, the others in registers
#pragma unroll
    for (int x = 0; x < 2 * KT; x++) {
        const auto K = Row<T>::natural(kb, kat, h, x), Q = Row<T>::natural(qb, qat, h, x);
        mm<IN>(kk, K, K);
        mm<IN>(kq, K, Q);                                      // k_j.q_i, lane i
        if (TRAIN) mm<IN>(qk, Q, K);                           // q_i.k_j, lane j
    }
    // P in rows of i, M into LDS, P^T in rows of j
    f32x16_t P, PT;
#pragma unroll
    for (int g4 = 0; g4 < 4; g4++) {
        const int j0 = 8 * g4 + 4 * h;
        const f32x4_t ghi = *reinterpret_cast<const f32x4_t *>(sc + kScHi + j0);
        const f32x4_t glo = *reinterpret_cast<const f32x4_t *>(sc + kScLo + j0);
        f32x4_t m;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int j = j0 + e, r = 4 * g4 + e;
            // the rows up to the lane's, and (transposed) from the lane's on
            const float d = j <= c ? exp_of(hi - ghi[e], lo - glo[e]) : 0.f;
            P[r] = j <= c ? A.scale * d * kq[r] : 0.f;
            m[e] = j < c ? b * d * kk[r] : 0.f;
            if (TRAIN) PT[r] = j >= c ? A.scale * exp_of(ghi[e] - hi, glo[e] - lo) * qk[r] : 0.f;
        }
        *reinterpret_cast<f32x4_t *>(lds + c * kPitch + j0) = m;
    }
#pragma unroll
    for (int kc = 0; kc < 2; kc++) {
        store_frag<OUT>(rec + Rec<T>::p, kc, operand<OUT>(P, kc));
        if (TRAIN) store_frag<ST>(rec + Rec<T>::pt, kc, operand<ST>(PT, kc));
    }
    wave_sync();
    // N by forward substitution, a column a lane: n_i = [i = c] - sum over j < i of M_ij n_j
    float nn[32];
#pragma unroll
    for (int i = 0; i < 32; i++) {
        float x = i == c ? 1.f : 0.f;
#pragma unroll
        for (int j4 = 0; j4 < (i + 3) / 4; j4++) {
            const f32x4_t m = *reinterpret_cast<const f32x4_t *>(lds + i * kPitch + 4 * j4);
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (4 * j4 + e < i) x = fmaf(-m[e], nn[4 * j4 + e], x);
        }
        nn[i] = x;
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < 16; i++) lds[(16 * h + i) * kPitch + c] = h ? nn[16 + i] : nn[i];
    wave_sync();
#pragma unroll
    for (int kc = 0; kc < 2; kc++) {
        float f[8];
        const f32x4_t x = *reinterpret_cast<const f32x4_t *>(lds + c * kPitch + 16 * kc + 4 * h);
        const f32x4_t y = *reinterpret_cast<const f32x4_t *>(lds + c * kPitch + 16 * kc + 8 + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            f[e] = x[e];
            f[4 + e] = y[e];
        }
        store_frag<ST>(rec + Rec<T>::n, kc, split8<ST>(f));
        if (TRAIN) {
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const int i = 16 * kc + 8 * (e >> 2) + (e & 3);
                f[e] = h ? nn[i + 4] : nn[i];
            }
            store_frag<ST>(rec + Rec<T>::nt, kc, split8<ST>(f));
        }
    }
    // K^T and Q^T: a lane has one element of every row
    if (head % A.group) return;
    char *recT = A.recT + ((int64_t)tile * A.key_heads + key) * A.recT_size;
#pragma unroll
    for (int side = 0; side < (TRAIN ? 2 : 1); side++)
#pragma unroll
        for (int t = 0; t < KT; t++)
#pragma unroll
            for (int kc = 0; kc < 2; kc++) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int i = 16 * kc + 8 * (e >> 2) + (e & 3) + 4 * h;
                    const uint32_t at = (uint32_t)((i * (side ? A.qs : A.ks) + 32 * t + c) * sizeof(T));
                    f[e] = Row<T>::one(side ? qb : kb, kept >> i & 1 ? at : kOut);
                }
                store_frag<IN>(recT, (side * KT + t) * 2 + kc, split8<IN>(f));
            }
}

// ----------------------------------------------------------------- the walks

// One wavefront's part of a walk: 32 columns of one sample's and head's state.
struct Walk {
    int sample, head, key, slice, base, rows;
    bool any;
};

// Blocks of the slices of one state are neighbours on one XCD, whose L2 then holds the
// operands that they share.
__device__ __forceinline__ Walk walk_of(const DeltaArgs &A)
{
    Walk w;
    const int64_t x = blockIdx.x & 7, i = blockIdx.x >> 3;
    const int64_t pair = (i / A.slices) * 8 + x;
    w.any = pair < (int64_t)A.samples * A.heads;
    w.slice = (int)(i % A.slices);
    w.sample = (int)(pair / A.heads);
    w.head = (int)(pair % A.heads);
    w.key = w.head / A.group;
    w.base = w.rows = 0;
    if (w.any) {
        w.base = seg_edge(A.off, A.samples, A.n, w.sample + 1);
        w.rows = max(seg_edge(A.off, A.samples, A.n, w.sample + 2) - w.base, 0);
    }
    return w;
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1; }

// a scalar for each of a block's rows
__device__ __forceinline__ f32x16_t row_scalars(const float *p, int h)
{
    f32x16_t r;
#pragma unroll
    for (int g4 = 0; g4 < 4; g4++) {
        const f32x4_t x = *gp(reinterpret_cast<const f32x4_t *>(p + 8 * g4 + 4 * h));
#pragma unroll
        for (int e = 0; e < 4; e++) r[4 * g4 + e] = x[e];
    }
    return r;
}

// a block of rows [32, 32 columns]: a column a lane, `rows` a bit for each row that is read
// (or written); the others give zero
template <typename T>
__device__ __forceinline__ f32x16_t block_read(__amdgpu_buffer_rsrc_t r, int64_t stride, uint32_t rows, int h,
                                               uint32_t col)
{
    f32x16_t x;
    const uint32_t bits = rows >> (4 * h), at = col + (uint32_t)(4 * h * stride * sizeof(T));
#pragma unroll
    for (int i = 0; i < 16; i++)
        x[i] = Row<T>::one(r, (bits >> kk0(i) & 1) && col != kOut ? at + (uint32_t)(kk0(i) * stride * sizeof(T)) : kOut);
    return x;
}
template <typename T>
__device__ __forceinline__ void block_write(__amdgpu_buffer_rsrc_t r, int64_t stride, uint32_t rows, int h,
                                            uint32_t col, const f32x16_t &x)
{
    const uint32_t bits = rows >> (4 * h), at = col + (uint32_t)(4 * h * stride * sizeof(T));
#pragma unroll
    for (int i = 0; i < 16; i++)
        Row<T>::put(r, (bits >> kk0(i) & 1) && col != kOut ? at + (uint32_t)(kk0(i) * stride * sizeof(T)) : kOut, x[i]);
}

// states [dk, dv] in memory
template <int KT>
__device__ __forceinline__ void state_read(f32x16_t (&S)[KT], const float *p, int dk, int dv, int h, int col)
{
#pragma unroll
    for (int t = 0; t < KT; t++)
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const int r = 32 * t + kk0(i) + 4 * h;
            S[t][i] = p && r < dk && col < dv ? *gp(p + r * dv + col) : 0.f;
        }
}
template <int KT>
__device__ __forceinline__ void state_write(const f32x16_t (&S)[KT], float *p, int dk, int dv, int h, int col)
{
#pragma unroll
    for (int t = 0; t < KT; t++)
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const int r = 32 * t + kk0(i) + 4 * h;
            if (r < dk && col < dv) *gp(p + r * dv + col) = S[t][i];
        }
}

template <typename T, int KT, bool TRAIN>
__global__ __launch_bounds__(64) void delta_scan(DeltaArgs A)
{
    constexpr int IN = Prec<T>::IN, ST = Prec<T>::ST, OUT = Prec<T>::OUT;
    const Walk w = walk_of(A);
    if (!w.any) return;
    const int l = lane_id(), c = l & 31, h = l >> 5;
    const int col = 32 * w.slice + c, dvp = 32 * A.slices;
    const uint32_t colat = col < A.dv ? (uint32_t)(col * sizeof(T)) : kOut;
    const int64_t matrix = ((int64_t)w.sample * A.heads + w.head) * A.dk * A.dv;
    f32x16_t S[KT];
    state_read<KT>(S, A.state ? A.state + matrix : nullptr, A.dk, A.dv, h, col);
    const int tile0 = first_tile(w.base, w.sample);
    for (int r0 = 0; r0 < w.rows; r0 += kCut) {
        const int tile = tile0 + r0 / kCut;
        const int64_t row = (int64_t)w.base + r0;
        const int left = min(w.rows - r0, kCut);
        const char *rec = A.rec + ((int64_t)tile * A.heads + w.head) * A.rec_size;
        const char *recT = A.recT + ((int64_t)tile * A.key_heads + w.key) * A.recT_size;
        const float *sc = reinterpret_cast<const float *>(rec + Rec<T>::sc);
        const uint32_t kept = __float_as_uint(*gp(sc + kScKept)) & low_bits(left);
        const float end = *gp(sc + kScEnd);
        const auto qb = buffer<T>(A.q, row * A.qs + w.key * A.qh), kb = buffer<T>(A.k, row * A.ks + w.key * A.kh);
        const uint32_t qat = kept >> c & 1 ? (uint32_t)(c * A.qs * sizeof(T)) : kOut;
        const uint32_t kat = kept >> c & 1 ? (uint32_t)(c * A.ks * sizeof(T)) : kOut;
        const f32x16_t V = block_read<T>(buffer<T>(A.v, row * A.vs + w.head * A.vh), A.vs, kept, h, colat);
        if (TRAIN) {
            const auto sb = buffer<T>(A.s0, ((int64_t)tile * A.heads + w.head) * (32 * KT) * dvp);
#pragma unroll
            for (int t = 0; t < KT; t++)
                block_write<T>(sb, dvp, 0xFFFFFFFFu, h, (uint32_t)((32 * t * dvp + col) * sizeof(T)), S[t]);
        }
        f32x16_t X = zero16(), Y = zero16();
#pragma unroll
        for (int x = 0; x < 2 * KT; x++) {
            const Part<ST> sp = operand<ST>(S[x / 2], x % 2);
            mm<ST>(X, Row<T>::turned(kb, kat, h, x), sp);
            mm<OUT>(Y, Row<T>::turned(qb, qat, h, x), sp);
        }
        const f32x16_t b = row_scalars(sc + kScB, h), bg = row_scalars(sc + kScBG, h), sg = row_scalars(sc + kScG, h),
                       wt = row_scalars(sc + kScW, h);
        f32x16_t U = zero16();
#pragma unroll
        for (int i = 0; i < 16; i++) {
            X[i] = fmaf(b[i], V[i], -bg[i] * X[i]);
            Y[i] *= sg[i];
        }
#pragma unroll
        for (int kc = 0; kc < 2; kc++) mm<ST>(U, load_frag<ST>(rec + Rec<T>::n, kc), operand<ST>(X, kc));
#pragma unroll
        for (int kc = 0; kc < 2; kc++) mm<OUT>(Y, load_frag<OUT>(rec + Rec<T>::p, kc), operand<OUT>(U, kc));
        block_write<T>(buffer<T>(A.o, (row * A.heads + w.head) * A.dv), (int64_t)A.heads * A.dv, low_bits(left), h,
                       colat, Y);
        if (TRAIN)
            block_write<T>(buffer<T>(A.u, (row * A.heads + w.head) * dvp), (int64_t)A.heads * dvp, low_bits(left), h,
                           (uint32_t)(col * sizeof(T)), U);
#pragma unroll
        for (int i = 0; i < 16; i++) U[i] *= wt[i];
        Part<ST> up[2];
#pragma unroll
        for (int kc = 0; kc < 2; kc++) up[kc] = operand<ST>(U, kc);
#pragma unroll
        for (int t = 0; t < KT; t++) {
#pragma unroll
            for (int i = 0; i < 16; i++) S[t][i] *= end;
#pragma unroll
            for (int kc = 0; kc < 2; kc++) mm<ST>(S[t], load_frag<IN>(recT, 2 * t + kc), up[kc]);
        }
    }
    state_write<KT>(S, A.last + matrix, A.dk, A.dv, h, col);
}

template <typename T, int KT>
__global__ __launch_bounds__(64) void delta_back(DeltaArgs A)
{
    constexpr int IN = Prec<T>::IN, ST = Prec<T>::ST;
    const Walk w = walk_of(A);
    if (!w.any) return;
    const int l = lane_id(), c = l & 31, h = l >> 5;
    const int col = 32 * w.slice + c, dvp = 32 * A.slices;
    const uint32_t colat = col < A.dv ? (uint32_t)(col * sizeof(T)) : kOut;
    const int64_t matrix = ((int64_t)w.sample * A.heads + w.head) * A.dk * A.dv;
    f32x16_t E[KT];
    state_read<KT>(E, A.dlast ? A.dlast + matrix : nullptr, A.dk, A.dv, h, col);
    const int tile0 = first_tile(w.base, w.sample);
    for (int r0 = w.rows > 0 ? (w.rows - 1) / kCut * kCut : -1; r0 >= 0; r0 -= kCut) {
        const int tile = tile0 + r0 / kCut;
        const int64_t row = (int64_t)w.base + r0;
        const int left = min(w.rows - r0, kCut);
        const char *rec = A.rec + ((int64_t)tile * A.heads + w.head) * A.rec_size;
        const char *recT = A.recT + ((int64_t)tile * A.key_heads + w.key) * A.recT_size;
        const float *sc = reinterpret_cast<const float *>(rec + Rec<T>::sc);
        const uint32_t kept = __float_as_uint(*gp(sc + kScKept)) & low_bits(left);
        const float end = *gp(sc + kScEnd);
        const auto kb = buffer<T>(A.k, row * A.ks + w.key * A.kh);
        const uint32_t kat = kept >> c & 1 ? (uint32_t)(c * A.ks * sizeof(T)) : kOut;
        f32x16_t D = block_read<T>(buffer<T>(A.dout, row * A.ds + w.head * A.dh), A.ds, kept, h, colat);
        const auto eb = buffer<T>(A.e, ((int64_t)tile * A.heads + w.head) * (32 * KT) * dvp);
#pragma unroll
        for (int t = 0; t < KT; t++)
            block_write<T>(eb, dvp, 0xFFFFFFFFu, h, (uint32_t)((32 * t * dvp + col) * sizeof(T)), E[t]);
        f32x16_t X = zero16();
#pragma unroll
        for (int x = 0; x < 2 * KT; x++) mm<ST>(X, Row<T>::turned(kb, kat, h, x), operand<ST>(E[x / 2], x % 2));
        const f32x16_t b = row_scalars(sc + kScB, h), bg = row_scalars(sc + kScBG, h), sg = row_scalars(sc + kScG, h),
                       wt = row_scalars(sc + kScW, h);
#pragma unroll
        for (int i = 0; i < 16; i++) X[i] *= wt[i];
#pragma unroll
        for (int kc = 0; kc < 2; kc++) mm<ST>(X, load_frag<ST>(rec + Rec<T>::pt, kc), operand<IN>(D, kc));
        f32x16_t Z = zero16();
#pragma unroll
        for (int kc = 0; kc < 2; kc++) mm<ST>(Z, load_frag<ST>(rec + Rec<T>::nt, kc), operand<ST>(X, kc));
        block_write<T>(buffer<T>(A.z, (row * A.heads + w.head) * dvp), (int64_t)A.heads * dvp, low_bits(left), h,
                       (uint32_t)(col * sizeof(T)), Z);
#pragma unroll
        for (int i = 0; i < 16; i++) {
            X[i] = b[i] * Z[i];
            Z[i] *= -bg[i];
            D[i] *= sg[i];
        }
        block_write<T>(buffer<T>(A.dv_, (row * A.heads + w.head) * A.dv), (int64_t)A.heads * A.dv, low_bits(left), h,
                       colat, X);
        Part<ST> zp[2], dp[2];
#pragma unroll
        for (int kc = 0; kc < 2; kc++) {
            zp[kc] = operand<ST>(Z, kc);
            dp[kc] = operand<ST>(D, kc);
        }
#pragma unroll
        for (int t = 0; t < KT; t++) {
#pragma unroll
            for (int i = 0; i < 16; i++) E[t][i] *= end;
#pragma unroll
            for (int kc = 0; kc < 2; kc++) {
                mm<ST>(E[t], load_frag<IN>(recT, 2 * t + kc), zp[kc]);
                mm<ST>(E[t], load_frag<IN>(recT, 2 * (KT + t) + kc), dp[kc]);
            }
        }
    }
    if (A.dstate) state_write<KT>(E, A.dstate + matrix, A.dk, A.dv, h, col);
}

// ----------------------------------------------------------------- gradients

template <typename T>
__device__ __forceinline__ float dot_parts(const Part<1> &a, const Part<1> &b)
{
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 4; j++)
        s += bf16_lo(a.p[0][j]) * bf16_lo(b.p[0][j]) + bf16_hi(a.p[0][j]) * bf16_hi(b.p[0][j]);
    return s;
}
template <typename T>
__device__ __forceinline__ float dot_parts(const Part<3> &a, const Part<3> &b)
{
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        s += (bf16_lo(a.p[0][j]) + bf16_lo(a.p[1][j]) + bf16_lo(a.p[2][j])) *
             (bf16_lo(b.p[0][j]) + bf16_lo(b.p[1][j]) + bf16_lo(b.p[2][j]));
        s += (bf16_hi(a.p[0][j]) + bf16_hi(a.p[1][j]) + bf16_hi(a.p[2][j])) *
             (bf16_hi(b.p[0][j]) + bf16_hi(b.p[1][j]) + bf16_hi(b.p[2][j]));
    }
    return s;
}

// One chunk and key head: wavefront w makes columns 32 w .. of dq and dk, all of them the
// products of rows with rows, the first dgate and dbeta.
template <typename T, int KT>
__global__ __launch_bounds__(64 * KT) void delta_grads(DeltaArgs A)
{
    constexpr int IN = Prec<T>::IN, OUT = Prec<T>::OUT;
    __shared__ float red[KT][3][32];
    const int tile = blockIdx.x, key = blockIdx.y;
    const int wave = uniform((int)(threadIdx.x >> 6)), l = lane_id(), c = l & 31, h = l >> 5;
    const SegTile s = seg_find<kCut>(A.off, A.n, nullptr, 0, A.samples, 1, tile);
    if (s.row0 >= s.rows) return;
    const int left = min(s.rows - s.row0, kCut), dvp = 32 * A.slices;
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
    const auto qb = buffer<T>(A.q, row * A.qs + key * A.qh), kb = buffer<T>(A.k, row * A.ks + key * A.kh);
    const uint32_t qat = keep ? (uint32_t)(c * A.qs * sizeof(T)) : kOut;
    const uint32_t kat = keep ? (uint32_t)(c * A.ks * sizeof(T)) : kOut;
    f32x16_t kk = zero16(), kq = zero16(), qk = zero16();
#pragma unroll
    for (int x = 0; x < 2 * KT; x++) {
        const auto K = Row<T>::natural(kb, kat, h, x), Q = Row<T>::natural(qb, qat, h, x);
        mm<IN>(kk, K, K);
        mm<IN>(kq, K, Q);
        mm<IN>(qk, Q, K);
    }
    float fq[16], fk[16];                                // the row's own elements of this wavefront's columns
#pragma unroll
    for (int x = 0; x < 2; x++) {
        Row<T>::floats(qb, qat, h, 2 * wave + x, fq + 8 * x);
        Row<T>::floats(kb, kat, h, 2 * wave + x, fk + 8 * x);
    }
    const char *recT = A.recT + ((int64_t)tile * A.key_heads + key) * A.recT_size;
    f32x16_t dq = zero16(), dk = zero16();               // transposed: a row a lane
    for (int g = 0; g < A.group; g++) {
        const int head = key * A.group + g;
        const char *rec = A.rec + ((int64_t)tile * A.heads + head) * A.rec_size;
        const float *sc = reinterpret_cast<const float *>(rec + Rec<T>::sc);
        const float b = *gp(sc + kScB + c), bg = *gp(sc + kScBG + c), sg = *gp(sc + kScG + c), wt = *gp(sc + kScW + c),
                    hi = *gp(sc + kScHi + c), lo = *gp(sc + kScLo + c), end = *gp(sc + kScEnd);
        const int64_t m0 = (((int64_t)tile * A.heads + head) * (32 * KT) + 32 * wave) * dvp;
        const auto sb = buffer<T>(A.s0, m0), eb = buffer<T>(A.e, m0);
        const auto ub = buffer<T>(A.u, (row * A.heads + head) * dvp), zb = buffer<T>(A.z, (row * A.heads + head) * dvp);
        const auto ob = buffer<T>(A.dop, row * A.dps + head * A.dph);
        const uint32_t mat = (uint32_t)(c * dvp * sizeof(T));
        const uint32_t uat = keep ? (uint32_t)((int64_t)c * A.heads * dvp * sizeof(T)) : kOut;
        const uint32_t oat = keep ? (uint32_t)(c * A.dps * sizeof(T)) : kOut;
        f32x16_t t1 = zero16(), t2 = zero16(), t3 = zero16();
        f32x16_t ud = zero16(), du = zero16(), uz = zero16(), zu = zero16();
        float inner = 0.f;
        for (int x = 0; x < 2 * A.slices; x++) {
            const auto S = Row<T>::natural(sb, mat, h, x), E = Row<T>::natural(eb, mat, h, x),
                       U = Row<T>::natural(ub, uat, h, x), Z = Row<T>::natural(zb, uat, h, x),
                       D = Row<T>::natural(ob, oat, h, x);
            mm<IN>(t1, S, D);
            mm<IN>(t2, S, Z);
            mm<IN>(t3, E, U);
            mm<IN>(ud, U, D);                            // u_j.dO_i, lane i
            mm<IN>(du, D, U);                            // dO_i.u_j, lane j
            mm<IN>(uz, U, Z);
            mm<IN>(zu, Z, U);
            inner += dot_parts<T>(S, E);
        }
        // lane x: what k_y (or q_y) is taken with, in register y
        f32x16_t forq, fork, fromq;
        float across = 0.f, own = 0.f;                   // row sum of H less column sum; z.u of the row
#pragma unroll
        for (int g4 = 0; g4 < 4; g4++) {
            const int y0 = 8 * g4 + 4 * h;
            const f32x4_t yhi = *gp(reinterpret_cast<const f32x4_t *>(sc + kScHi + y0));
            const f32x4_t ylo = *gp(reinterpret_cast<const f32x4_t *>(sc + kScLo + y0));
            const f32x4_t yb = *gp(reinterpret_cast<const f32x4_t *>(sc + kScB + y0));
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int y = y0 + e, r = 4 * g4 + e;
                const bool before = y < c, after = y > c;
                const float d = exp_of(before ? hi - yhi[e] : yhi[e] - hi, before ? lo - ylo[e] : ylo[e] - lo);
                const float D = y <= c ? A.scale * d * ud[r] : 0.f;        // D_xy
                const float DT = y >= c ? A.scale * d * du[r] : 0.f;       // D_yx
                const float B = before ? -b * d * uz[r] : after ? -yb[e] * d * zu[r] : 0.f;   // B_xy or B_yx
                forq[r] = D;
                fromq[r] = DT;
                fork[r] = B;
                if (y == c) own += uz[r];
                across += before ? fmaf(D, kq[r], B * kk[r]) : after ? -fmaf(DT, qk[r], B * kk[r]) : 0.f;
            }
        }
#pragma unroll
        for (int kc = 0; kc < 2; kc++) {
            const Part<IN> kt = load_frag<IN>(recT, 2 * wave + kc), qt = load_frag<IN>(recT, 2 * (KT + wave) + kc);
            mm<OUT>(dq, kt, operand<OUT>(forq, kc));
            mm<OUT>(dk, kt, operand<OUT>(fork, kc));
            mm<OUT>(dk, qt, operand<OUT>(fromq, kc));
        }
        float dots = 0.f, writes = 0.f;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float x = sg * t1[i], y = -bg * t2[i], z = wt * t3[i];
            dq[i] += x;
            dk[i] += y + z;
            dots += fmaf(x, fq[i], y * fk[i]);
            writes = fmaf(z, fk[i], writes);
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
            float from = both(across), into = 0.f, state = 0.f;
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
            own = both(own);
            if (valid && h == 0) {
                float dg = 0.f, db = 0.f;
                if (keep) {
                    const float gate = Row<T>::get1(static_cast<const T *>(A.gate) + (row + c) * A.gs + head);
                    const float beta = Row<T>::get1(static_cast<const T *>(A.beta) + (row + c) * A.bs + head);
                    // a gate that forgets all has none, whatever the sums' rounding leaves
                    dg = expf(-gate) == INFINITY ? 0.f : (suffix + prefix + end * state) / (1.f + expf(gate));
                    db = own / (1.f + expf(beta));
                }
                Row<T>::put1(static_cast<T *>(A.dgate) + (row + c) * A.heads + head, dg);
                Row<T>::put1(static_cast<T *>(A.dbeta) + (row + c) * A.heads + head, db);
            }
        }
        __syncthreads();
    }
    if (!valid) return;
    const int64_t at = ((row + c) * A.key_heads + key) * A.dk;
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
                Row<T>::put4(static_cast<T *>(A.dq) + at + x0, a);
                Row<T>::put4(static_cast<T *>(A.dk_) + at + x0, b);
            }
        } else {
            for (int e = 0; e < 4; e++)
                if (x0 + e < A.dk) {
                    Row<T>::put1(static_cast<T *>(A.dq) + at + x0 + e, a[e]);
                    Row<T>::put1(static_cast<T *>(A.dk_) + at + x0 + e, b[e]);
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
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n * heads * padded) return;
    const int c = (int)(i % padded);
    const int64_t rh = i / padded;
    const int64_t r = rh / heads, h = rh % heads;
    *gp(y + i) = c < d ? *gp(x + r * xs + h * xh + c) : T(0);
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
    size_t rec, recT;                        // bytes of a record
    size_t recs, recTs, states, us;          // bytes of all records, states and U
    size_t q, k, o;                          // bytes of packed rows, 0 where they are read in place
    size_t saved, forward, backward;
};

DeltaPlan delta_plan(const emb_delta *d, bool train, bool any_layout)
{
    DeltaPlan p{};
    p.el = d->dtype == EMB_BF16 ? 2 : 4;
    p.kt = (d->dk + 31) / 32;
    p.slices = (d->dv + 31) / 32;
    p.tiles = seg_tiles(d->n, d->samples, 1, kCut);
    const bool bf = d->dtype == EMB_BF16;
    p.rec = train ? (bf ? Rec<uint16_t>::whole : Rec<float>::whole) : (bf ? Rec<uint16_t>::small : Rec<float>::small);
    p.recT = (size_t)p.kt * (train ? 2 : 1) * 2 * (bf ? 1 : 3) * 1024;
    p.recs = pad256((size_t)p.tiles * d->heads * p.rec);
    p.recTs = pad256((size_t)p.tiles * d->key_heads * p.recT);
    p.states = pad256((size_t)p.tiles * d->heads * p.kt * 32 * p.slices * 32 * p.el);
    p.us = pad256((size_t)d->n * d->heads * p.slices * 32 * p.el);
    const size_t packed = pad256((size_t)d->n * d->key_heads * p.kt * 32 * p.el);
    p.q = any_layout || !rows_ready(d->q, d->q_stride, d->q_head_stride, d->dk, p.el) ? packed : 0;
    p.k = any_layout || !rows_ready(d->k, d->k_stride, d->k_head_stride, d->dk, p.el) ? packed : 0;
    p.o = p.us;
    p.saved = p.recs + p.recTs + p.states + p.us;
    p.forward = (train ? 0 : p.recs + p.recTs) + p.q + p.k;
    p.backward = p.states + p.us + p.q + p.k + p.o;
    return p;
}

emb_status delta_launched()
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(EMB_ERR_HIP, std::string("delta rule launch: ") + hipGetErrorString(e));
    return EMB_OK;
}

template <typename T>
void delta_pack_rows(const void *x, int64_t xs, int64_t xh, void *y, int64_t n, int heads, int d, int padded, hipStream_t st)
{
    const int64_t blocks = (n * heads * padded + 255) / 256;
    if (blocks)
        hipLaunchKernelGGL((delta_pack<T>), dim3((unsigned)blocks), dim3(256), 0, st, static_cast<const T *>(x), xs, xh,
                           static_cast<T *>(y), n, heads, d, padded);
}

// q and k as the kernels read them: in place, or packed into *ws, which moves on
template <typename T>
void delta_rows(const emb_delta *d, const DeltaPlan &p, DeltaArgs &A, char *&ws, hipStream_t st)
{
    if (p.q) {
        delta_pack_rows<T>(d->q, d->q_stride, d->q_head_stride, ws, d->n, d->key_heads, d->dk, 32 * p.kt, st);
        A.q = ws;
        A.qh = 32 * p.kt;
        A.qs = A.qh * d->key_heads;
        ws += p.q;
    }
    if (p.k) {
        delta_pack_rows<T>(d->k, d->k_stride, d->k_head_stride, ws, d->n, d->key_heads, d->dk, 32 * p.kt, st);
        A.k = ws;
        A.kh = 32 * p.kt;
        A.ks = A.kh * d->key_heads;
        ws += p.k;
    }
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
    A.recT_size = (int64_t)p.recT;
    return A;
}

// records, states and U in the buffer that the forward leaves for the backward
void delta_saved(const DeltaPlan &p, DeltaArgs &A, char *saved)
{
    A.rec = saved;
    A.recT = saved + p.recs;
    A.s0 = saved + p.recs + p.recTs;
    A.u = saved + p.recs + p.recTs + p.states;
}

int64_t walk_blocks(const emb_delta *d, const DeltaPlan &p)
{
    const int64_t pairs = ((int64_t)d->samples * d->heads + 7) / 8 * 8;
    return pairs * p.slices;
}

emb_status delta_sizes(const emb_delta *d, const DeltaPlan &p)
{
    // a launch's threads in one dimension are counted in 32 bits
    const int64_t most = (int64_t(1) << 32) - 1, packed = d->n * d->heads * 128;
    if (p.tiles > most / (64 * 4) || walk_blocks(d, p) > most / 64 || packed > most)
        return fail(EMB_ERR_UNSUPPORTED, "delta rule: too many rows, samples and heads for one launch");
    return EMB_OK;
}

template <typename T, int KT>
void delta_forward_launch(const DeltaArgs &A, int64_t tiles, int64_t walks, bool train, hipStream_t st)
{
    const dim3 all((unsigned)tiles, (unsigned)A.heads), walk((unsigned)walks), block(64);
    if (train) {
        hipLaunchKernelGGL((delta_prepare<T, KT, true>), all, block, 0, st, A);
        if (walks) hipLaunchKernelGGL((delta_scan<T, KT, true>), walk, block, 0, st, A);
    } else {
        hipLaunchKernelGGL((delta_prepare<T, KT, false>), all, block, 0, st, A);
        if (walks) hipLaunchKernelGGL((delta_scan<T, KT, false>), walk, block, 0, st, A);
    }
}

template <typename T, int KT>
void delta_backward_launch(const DeltaArgs &A, int64_t tiles, int64_t walks, hipStream_t st)
{
    if (walks) hipLaunchKernelGGL((delta_back<T, KT>), dim3((unsigned)walks), dim3(64), 0, st, A);
    hipLaunchKernelGGL((delta_grads<T, KT>), dim3((unsigned)tiles, (unsigned)A.key_heads), dim3(64 * KT), 0, st, A);
}

template <typename T>
void delta_forward_any(int kt, const DeltaArgs &A, int64_t tiles, int64_t walks, bool train, hipStream_t st)
{
    if (kt == 1) delta_forward_launch<T, 1>(A, tiles, walks, train, st);
    else if (kt == 2) delta_forward_launch<T, 2>(A, tiles, walks, train, st);
    else if (kt == 3) delta_forward_launch<T, 3>(A, tiles, walks, train, st);
    else delta_forward_launch<T, 4>(A, tiles, walks, train, st);
}

template <typename T>
void delta_backward_any(int kt, const DeltaArgs &A, int64_t tiles, int64_t walks, hipStream_t st)
{
    if (kt == 1) delta_backward_launch<T, 1>(A, tiles, walks, st);
    else if (kt == 2) delta_backward_launch<T, 2>(A, tiles, walks, st);
    else if (kt == 3) delta_backward_launch<T, 3>(A, tiles, walks, st);
    else delta_backward_launch<T, 4>(A, tiles, walks, st);
}

}  // namespace

extern "C" emb_status emb_delta_query(const emb_delta *d, int32_t training, size_t *saved_bytes, size_t *forward_bytes,
                                      size_t *backward_bytes)
{
    if (!d) return fail(EMB_ERR_INVALID_ARG, "delta rule descriptor is NULL");
    const emb_status s = delta_check(d);
    if (s != EMB_OK) return s;
    if (!saved_bytes || !forward_bytes || !backward_bytes)
        return fail(EMB_ERR_INVALID_ARG, "delta rule: output pointers must be given");
    *saved_bytes = training ? delta_plan(d, true, false).saved : 0;
    *forward_bytes = delta_plan(d, training != 0, false).forward;
    // the tensors that the backward gets may lie otherwise than the forward's did
    *backward_bytes = training ? delta_plan(d, true, true).backward : 0;
    return EMB_OK;
}

extern "C" emb_status emb_delta_forward(const emb_delta *d, void *o, float *last, void *saved, void *workspace,
                                        size_t workspace_bytes, void *stream)
{
    if (!d) return fail(EMB_ERR_INVALID_ARG, "delta rule descriptor is NULL");
    emb_status s = delta_check(d);
    if (s == EMB_OK) s = delta_pointers(d);
    if (s != EMB_OK) return s;
    const DeltaPlan p = delta_plan(d, saved != nullptr, false);
    if ((d->n && !o) || (d->samples && !last) || !aligned(o, p.el) || !aligned(last, 4) || !aligned(saved, 256))
        return fail(EMB_ERR_INVALID_ARG, "delta rule: o and last must be given and aligned, saved to 256 bytes");
    if (workspace_bytes < p.forward || (p.forward && (!workspace || !aligned(workspace, 256))))
        return fail(EMB_ERR_WORKSPACE, "delta rule: the workspace is smaller than the query returned, or not 256-byte aligned");
    s = delta_sizes(d, p);
    if (s != EMB_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    DeltaArgs A = delta_args(d, p);
    A.o = o;
    A.last = last;
    char *ws = static_cast<char *>(workspace);
    if (saved) delta_saved(p, A, static_cast<char *>(saved));
    else {
        A.rec = ws;
        A.recT = ws + p.recs;
        ws += p.recs + p.recTs;
    }
    const int64_t walks = walk_blocks(d, p);
    if (d->dtype == EMB_BF16) {
        delta_rows<uint16_t>(d, p, A, ws, st);
        delta_forward_any<uint16_t>(p.kt, A, p.tiles, walks, saved != nullptr, st);
    } else {
        delta_rows<float>(d, p, A, ws, st);
        delta_forward_any<float>(p.kt, A, p.tiles, walks, saved != nullptr, st);
    }
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
    DeltaPlan p = delta_plan(d, true, false);
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
    if (rows_ready(dout, dout_stride, dout_head_stride, d->dv, p.el)) p.o = 0;
    p.backward = p.states + p.us + p.q + p.k + p.o;
    if (workspace_bytes < p.backward || (p.backward && (!workspace || !aligned(workspace, 256))))
        return fail(EMB_ERR_WORKSPACE, "delta rule: the workspace is smaller than the query returned, or not 256-byte aligned");
    s = delta_sizes(d, p);
    if (s != EMB_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    DeltaArgs A = delta_args(d, p);
    delta_saved(p, A, const_cast<char *>(static_cast<const char *>(saved)));
    char *ws = static_cast<char *>(workspace);
    A.e = ws;
    A.z = ws + p.states;
    ws += p.states + p.us;
    A.dout = A.dop = dout;
    A.ds = A.dps = dout_stride;
    A.dh = A.dph = dout_head_stride;
    A.dlast = dlast;
    A.dq = dq;
    A.dk_ = dk;
    A.dv_ = dv;
    A.dgate = dgate;
    A.dbeta = dbeta;
    A.dstate = dstate;
    A.vec = d->dk % 4 == 0 && aligned(dq, 4 * p.el) && aligned(dk, 4 * p.el);
    const int64_t walks = walk_blocks(d, p);
    const bool bf = d->dtype == EMB_BF16;
    if (bf) delta_rows<uint16_t>(d, p, A, ws, st);
    else delta_rows<float>(d, p, A, ws, st);
    if (p.o) {
        if (bf) delta_pack_rows<uint16_t>(dout, dout_stride, dout_head_stride, ws, d->n, d->heads, d->dv, 32 * p.slices, st);
        else delta_pack_rows<float>(dout, dout_stride, dout_head_stride, ws, d->n, d->heads, d->dv, 32 * p.slices, st);
        A.dop = ws;
        A.dph = 32 * p.slices;
        A.dps = A.dph * d->heads;
    }
    if (bf) delta_backward_any<uint16_t>(p.kt, A, p.tiles, walks, st);
    else delta_backward_any<float>(p.kt, A, p.tiles, walks, st);
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
