// rotary.hip -- rotary positions: each pair of a head's elements turned by an angle that
// grows with the row's position,
//   (a, b) -> scale (a cos t - b sin t, b cos t + a sin t),  t = pos * frequency[pair],
// in one launch for queries and keys; the gradient is the turn back.  Pairs are (j, j + pairs)
// or neighbours (2 j, 2 j + 1) of the head's first 2 pairs elements; the others are copied.
//
// Angles.  Positions are int32 and may be elapsed seconds, so pos * frequency in fp32 would
// lose the angle.  A frequency becomes a 64-bit fraction of a turn, whose product with the
// position wraps at whole turns by itself: what is left is exact but for 2^-64 |pos| turns (7e-10
// radians at most).  Its top 32 bits split into a quadrant and an angle within +-pi/4, where the
// Taylor series of sine (to the 9th power) and cosine (to the 10th) are within 3e-9 of them.
//
// The bound is reading and writing every element once.  A workgroup takes some rows, makes
// their cosines and sines once in LDS, and turns all heads with them, 16 bytes a lane.
// 28528 rows of 8 heads of 128 in bf16: 21 us (117 MB, 5.6 TB/s); 65838 rows of 3 and 6 heads, 24
// of 40 elements, in fp32: 16.7 us (64 MB, 3.8 TB/s).
#include <cmath>
#include <string>

#include "sequence.h"

namespace emb {

constexpr int kRotaryDim = 1024;       // largest head
constexpr int kRotaryTable = 1024;     // angles of a workgroup
constexpr int kRotaryThreads = 256;

struct RotarySide {
    const void *x;
    void *y;
    const int32_t *pos;
    int64_t n, xs, xh;
    int32_t heads;
};

struct RotaryArgs {
    RotarySide side[2];
    int64_t blocks0;                   // workgroups of the first side
    const double *freq;
    int32_t dim, pairs, rows;          // rows of a workgroup
    int32_t shift;                     // 2^shift threads side by side make a row's angles
    int32_t items, magic;              // items of a head, ceil(2^32 / items) or 0 for one
    float scale, sign;
};

// a frequency (radians a step) as a fraction of a turn in units of 2^-64; 1 / (2 pi) in two doubles.
// Of its magnitude: hi less its whole turns is exact for hi >= 0 alone, and has to be of hi as it is
// rounded (contracted into the product it would hold what lo holds).
__device__ __forceinline__ uint64_t turn_of(double f)
{
#pragma clang fp contract(off)
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
    const double m = fabs(f), hi = m * kHi, lo = fma(m, kHi, -hi) + m * kLo;
    const double part = hi - floor(hi);
    const uint64_t turn = (uint64_t)rint(part * 0x1p64) + (uint64_t)(int64_t)rint(lo * 0x1p64);
    return f < 0. ? 0 - turn : turn;
}

__device__ __forceinline__ void turned(uint64_t turn, int pos, float &c, float &s)
{
    const uint64_t t = turn * (uint64_t)(int64_t)pos;
    const uint32_t a = (uint32_t)((t + 0x80000000ull) >> 32);
    const uint32_t quarter = (a + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(a - (quarter << 30)) * 1.4629180792671596e-09f;   // 2 pi / 2^32
    const float z = x * x;
    const float sn = x * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), 1.f);
    const float cs = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
    const float c1 = quarter & 1 ? -sn : cs, s1 = quarter & 1 ? cs : sn;
    c = quarter & 2 ? -c1 : c1;
    s = quarter & 2 ? -s1 : s1;
}

// i / d for i < 2^16 with magic = ceil(2^32 / d) (0: d is one)
__device__ __forceinline__ int over(int i, int magic) { return magic ? (int)__umulhi((uint32_t)i, (uint32_t)magic) : i; }

// an element as a number and back
__device__ __forceinline__ float open1(uint16_t x) { return bf16_lo((uint32_t)x); }
__device__ __forceinline__ float open1(float x) { return x; }
template <typename T>
__device__ __forceinline__ T shut1(float x)
{
    if constexpr (sizeof(T) == 2) return bf16_rne(x);
    else return x;
}

// WIDE: heads in pieces of 16 bytes, else pair by pair; HALF: pairs (j, j + pairs).
template <typename T, bool WIDE, bool HALF>
__global__ __launch_bounds__(kRotaryThreads) void rotary_turn(RotaryArgs A)
{
    typedef Piece<T> P;
    constexpr int E = P::E;
    __shared__ __attribute__((aligned(16))) float cs[kRotaryTable], sn[kRotaryTable];
    const bool second = blockIdx.x >= A.blocks0;
    const RotarySide &S = A.side[second];
    const int64_t row0 = (int64_t)(blockIdx.x - (second ? A.blocks0 : 0)) * A.rows;
    const int rows = (int)min((int64_t)A.rows, S.n - row0);
    // a pair a thread, as many rows side by side as there is room for (a thread that makes all rows
    // of its pair: 20.5 us at least for the second example above, 14.8 so)
    for (int p = threadIdx.x & ((1 << A.shift) - 1); p < A.pairs; p += 1 << A.shift) {
        const double f = *gp(A.freq + p);
        const bool far = !(fabs(f) <= 1e9);
        const uint64_t turn = far ? 0 : turn_of(f);
        for (int r = threadIdx.x >> A.shift; r < rows; r += kRotaryThreads >> A.shift) {
            float c, s;
            turned(turn, *gp(S.pos + row0 + r), c, s);
            cs[r * A.pairs + p] = far ? __builtin_nanf("") : A.scale * c;
            sn[r * A.pairs + p] = far ? __builtin_nanf("") : A.scale * A.sign * s;
        }
    }
    __syncthreads();
    const T *x = static_cast<const T *>(S.x);
    T *y = static_cast<T *>(S.y);
    const int per = A.items * S.heads;
    // a row at a time: what it has of items fills the workgroup, or several rows do together
    const int together = max(1, kRotaryThreads / per), mine = together > 1 ? threadIdx.x / per : 0;
    const int first = together > 1 ? threadIdx.x - mine * per : threadIdx.x;
    if (together > 1 && mine >= together) return;
    for (int r = mine; r < rows; r += together) {
        for (int it = first; it < per; it += kRotaryThreads) {
            const int head = over(it, A.magic), i = it - head * A.items;
            const T *src = x + (row0 + r) * S.xs + (int64_t)head * S.xh;
            T *dst = y + ((row0 + r) * S.heads + head) * A.dim;
            const float *c = cs + r * A.pairs, *s = sn + r * A.pairs;
            if (WIDE && HALF) {
                const int groups = A.pairs / E;
                if (i < groups) {
                    float a[E], b[E], u[E], v[E];
                    P::open(*gp(reinterpret_cast<const u32x4_t *>(src + i * E)), a);
                    P::open(*gp(reinterpret_cast<const u32x4_t *>(src + A.pairs + i * E)), b);
#pragma unroll
                    for (int e = 0; e < E; e++) {
                        const float cc = c[i * E + e], ss = s[i * E + e];
                        u[e] = a[e] * cc - b[e] * ss;
                        v[e] = b[e] * cc + a[e] * ss;
                    }
                    *gp(reinterpret_cast<u32x4_t *>(dst + i * E)) = P::shut(u);
                    *gp(reinterpret_cast<u32x4_t *>(dst + A.pairs + i * E)) = P::shut(v);
                } else {
                    const int at = 2 * A.pairs + (i - groups) * E;
                    *gp(reinterpret_cast<u32x4_t *>(dst + at)) = *gp(reinterpret_cast<const u32x4_t *>(src + at));
                }
            } else if (WIDE) {
                const u32x4_t w = *gp(reinterpret_cast<const u32x4_t *>(src + i * E));
                u32x4_t out = w;
                if (i * E < 2 * A.pairs) {
                    float a[E], u[E];
                    P::open(w, a);
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float cc = c[(i * E + e) / 2], ss = s[(i * E + e) / 2];
                        u[e] = a[e] * cc - a[e + 1] * ss;
                        u[e + 1] = a[e + 1] * cc + a[e] * ss;
                    }
                    out = P::shut(u);
                }
                *gp(reinterpret_cast<u32x4_t *>(dst + i * E)) = out;
            } else if (i < A.pairs) {
                const int at = HALF ? i : 2 * i, bt = HALF ? i + A.pairs : 2 * i + 1;
                const float a = open1(*gp(src + at)), b = open1(*gp(src + bt)), cc = c[i], ss = s[i];
                *gp(dst + at) = shut1<T>(a * cc - b * ss);
                *gp(dst + bt) = shut1<T>(b * cc + a * ss);
            } else {
                const int at = A.pairs + i;
                *gp(dst + at) = *gp(src + at);
            }
        }
    }
}

}  // namespace emb

using namespace emb;

namespace {

emb_status rotary_check(const emb_rotary *r)
{
    if (r->dtype != EMB_F32 && r->dtype != EMB_BF16) return fail(EMB_ERR_INVALID_ARG, "rotary: unknown dtype");
    if (r->layout != EMB_ROTARY_HALF && r->layout != EMB_ROTARY_INTERLEAVED)
        return fail(EMB_ERR_INVALID_ARG, "rotary: unknown layout");
    if (r->dim < 1 || r->pairs < 0 || 2 * (int64_t)r->pairs > r->dim)
        return fail(EMB_ERR_INVALID_ARG, "rotary: dim must be >= 1 and twice the pairs at most dim");
    if (r->dim > kRotaryDim) return fail(EMB_ERR_UNSUPPORTED, "rotary: dim must be <= 1024");
    if (!std::isfinite(r->scale)) return fail(EMB_ERR_INVALID_ARG, "rotary: scale must be finite");
    const size_t el = r->dtype == EMB_BF16 ? 2 : 4;
    if (r->pairs && (!r->frequencies || !aligned(r->frequencies, 8)))
        return fail(EMB_ERR_INVALID_ARG, "rotary: frequencies must be given");
    for (const emb_rotary_rows *s : {&r->q, &r->k}) {
        if (s->n < 0) return fail(EMB_ERR_INVALID_ARG, "rotary: n must be >= 0");
        if (!s->n) continue;
        if (s->heads < 1) return fail(EMB_ERR_INVALID_ARG, "rotary: heads must be >= 1");
        if (s->n > kRowsMost || (int64_t)s->heads * r->dim >= (1 << 16))
            return fail(EMB_ERR_UNSUPPORTED, "rotary: n must be <= 2^31 - 65536 and heads x dim < 2^16");
        if (s->stride < 0 || s->head_stride < 0) return fail(EMB_ERR_INVALID_ARG, "rotary: strides must be >= 0");
        if (!s->x || !s->y || !s->pos) return fail(EMB_ERR_INVALID_ARG, "rotary: x, y and pos must be given");
        if (!aligned(s->x, el) || !aligned(s->y, el) || !aligned(s->pos, 4))
            return fail(EMB_ERR_INVALID_ARG, "rotary: buffers must be aligned to their elements");
    }
    return EMB_OK;
}

int32_t magic_of(int d) { return d == 1 ? 0 : (int32_t)(uint32_t)(((int64_t(1) << 32) + d - 1) / d); }

template <typename T>
void rotary_launch(const RotaryArgs &A, bool wide, bool half, int64_t blocks, hipStream_t st)
{
    const dim3 grid((unsigned)blocks), block(kRotaryThreads);
    if (wide && half) hipLaunchKernelGGL((rotary_turn<T, true, true>), grid, block, 0, st, A);
    else if (wide) hipLaunchKernelGGL((rotary_turn<T, true, false>), grid, block, 0, st, A);
    else if (half) hipLaunchKernelGGL((rotary_turn<T, false, true>), grid, block, 0, st, A);
    else hipLaunchKernelGGL((rotary_turn<T, false, false>), grid, block, 0, st, A);
}

}  // namespace

extern "C" emb_status emb_rotary_turn(const emb_rotary *r, int32_t back, void *stream)
{
    if (!r) return fail(EMB_ERR_INVALID_ARG, "rotary descriptor is NULL");
    const emb_status s = rotary_check(r);
    if (s != EMB_OK) return s;
    if (!r->q.n && !r->k.n) return EMB_OK;
    const size_t el = r->dtype == EMB_BF16 ? 2 : 4;
    const int E = (int)(16 / el);
    const bool half = r->layout == EMB_ROTARY_HALF;
    // pieces of 16 bytes: no piece may hold elements of both members of a pair's halves, or of
    // what is turned and what is copied
    bool wide = r->dim % E == 0 && (half ? r->pairs % E == 0 : 2 * r->pairs % E == 0);
    for (const emb_rotary_rows *x : {&r->q, &r->k})
        if (x->n)
            wide = wide && aligned(x->x, 16) && aligned(x->y, 16) && x->stride * el % 16 == 0 && x->head_stride * el % 16 == 0;
    RotaryArgs A{};
    A.freq = r->frequencies;
    A.dim = r->dim;
    A.pairs = r->pairs;
    A.scale = r->scale;
    A.sign = back ? -1.f : 1.f;
    A.items = !wide ? r->dim - r->pairs : half ? (r->dim - r->pairs) / E : r->dim / E;
    A.magic = magic_of(A.items);
    // Rows of a workgroup: as many as the table of angles holds, fewer where that would leave
    // CUs without work.
    const int64_t all = r->q.n + r->k.n;
    int64_t rows = r->pairs ? kRotaryTable / r->pairs : 64;
    if (rows > 64) rows = 64;
    if (rows > (all + 511) / 512) rows = (all + 511) / 512;
    A.rows = (int32_t)rows;
    while (1 << A.shift < r->pairs && 1 << A.shift < kRotaryThreads) A.shift++;
    int64_t blocks = 0;
    for (int i = 0; i < 2; i++) {
        const emb_rotary_rows &x = i ? r->k : r->q;
        A.side[i] = RotarySide{x.x, x.y, x.pos, x.n, x.stride, x.head_stride, x.heads};
        if (i == 1) A.blocks0 = blocks;
        blocks += (x.n + rows - 1) / rows;
    }
    if (blocks > ((int64_t(1) << 32) - 1) / kRotaryThreads)
        return fail(EMB_ERR_UNSUPPORTED, "rotary: too many rows for one launch");
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (r->dtype == EMB_BF16) rotary_launch<uint16_t>(A, wide, half, blocks, st);
    else rotary_launch<float>(A, wide, half, blocks, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(EMB_ERR_HIP, std::string("rotary launch: ") + hipGetErrorString(e));
    return EMB_OK;
}
