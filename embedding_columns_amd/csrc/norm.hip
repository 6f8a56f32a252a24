// norm.hip -- layer norm over the last dimension of strided rows, forward and backward:
//   xh = (x - mean) r, r = 1 / sqrt(var + eps),  y = xh w + b
//   g = dy w,  dx = r (g - mean(g) - xh mean(g xh)),  dw = sum of dy xh, db = sum of dy over the rows
//
// The bound is reading x (and dy) and writing y (or dx) once: a row stays in registers, as it
// came, between its sums, which are taken of the centred values and in fp32.  A row is read by
// 1 .. 64 lanes (several rows share a wavefront) or by up to 16 wavefronts, 16 bytes a lane and
// piece.  Workgroups walk over rows, with weight and bias in registers (read again for each
// row they cost as much of the caches as x: 74 us for what takes 57) and, where registers last,
// the next row on its way; in the backward each keeps its share of dw and db in registers,
// leaves one row of them, and a second kernel adds these up in a fixed order.
//
// 140771 rows of 512 in bf16: forward 58 us (288 MB, 5.0 TB/s), backward 87 us (432 MB, 5.0 TB/s) and
// 5 us for the sums.  8191 of 5000 in fp32: 61 us (328 MB, 5.4 TB/s), 102 us (491 MB, 4.8 TB/s) and
// 6 us.  50 rows of 256: 3.8 us, a launch.
#include <cmath>
#include <string>

#include "sequence.h"

namespace emb {

constexpr int kNormChannels = 16384;

struct NormArgs {
    const void *x;
    int64_t xs, xi;                      // strides of the outer and the inner rows, in elements
    const float *w, *b;
    int64_t rows;
    int32_t inner, channels;
    int32_t lanes;                       // lanes of a row, a power of two (64 where it has whole wavefronts)
    float eps, part;                     // part: 1 / channels
    void *y;
    float *stats;                        // [rows, 2]: mean and r
    const void *dy;
    int64_t ds, di;
    void *dx;
    float *sums;                         // [workgroups, 2, channels]
    int32_t want_w, want_b;
};

// 16 bytes of a row that may start anywhere an element may
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Raw {
    u32x4_t w;
};

// Elements at .. at + E - 1 of a row, zeros behind its end.  WHOLE: rows are whole pieces.
template <typename T, bool WHOLE>
__device__ __forceinline__ u32x4_t piece_read(const T *row, int at, int channels)
{
    constexpr int E = Piece<T>::E;
    if (WHOLE ? at < channels : at + E <= channels) return gp(reinterpret_cast<const Raw<T> *>(row + at))->w;
    if (WHOLE) return u32x4_t{0, 0, 0, 0};
    union {
        u32x4_t w;
        T e[E];
    } u;
    u.w = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < E; i++)
        if (at + i < channels) u.e[i] = *gp(row + at + i);
    return u.w;
}
template <typename T, bool WHOLE>
__device__ __forceinline__ void piece_write(T *row, int at, int channels, const float *f)
{
    constexpr int E = Piece<T>::E;
    union {
        u32x4_t w;
        T e[E];
    } u;
    u.w = Piece<T>::shut(f);
    if (WHOLE || at + E <= channels) {
        gp(reinterpret_cast<Raw<T> *>(row + at))->w = u.w;
        return;
    }
#pragma unroll
    for (int i = 0; i < E; i++)
        if (at + i < channels) *gp(row + at + i) = u.e[i];
}
// the same of fp32 parameters; `fill` where there are none or behind the end
template <int E, bool WHOLE>
__device__ __forceinline__ void param_read(const float *p, int at, int channels, float fill, float *f)
{
#pragma unroll
    for (int i = 0; i < E; i++) f[i] = fill;
    if (!p) return;
    if (WHOLE ? at < channels : at + E <= channels) {
#pragma unroll
        for (int j = 0; j < E; j += 4) {
            const u32x4_t v = gp(reinterpret_cast<const Raw<float> *>(p + at + j))->w;
#pragma unroll
            for (int e = 0; e < 4; e++) f[j + e] = __uint_as_float(v[e]);
        }
    } else if (!WHOLE) {
#pragma unroll
        for (int i = 0; i < E; i++)
            if (at + i < channels) f[i] = *gp(p + at + i);
    }
}

// Sums over the lanes of a row, the same in all of them.  The wavefronts of a row meet in
// LDS, at `turn`'s place of two, so that one barrier a sum is enough.
template <bool MANY, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int lanes, float (*meet)[16][N], int turn)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1)
        if (MANY || m < lanes)
#pragma unroll
            for (int i = 0; i < N; i++) v[i] += __shfl_xor(v[i], m, 64);
    if (!MANY) return;
    if (lane_id() == 0)
#pragma unroll
        for (int i = 0; i < N; i++) meet[turn][threadIdx.x >> 6][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; i++) {
        float s = 0.f;
        for (int w = 0; w < (int)(blockDim.x >> 6); w++) s += meet[turn][w][i];
        v[i] = s;
    }
}

__device__ __forceinline__ int64_t norm_at(int64_t r, int inner, int64_t so, int64_t si)
{
    if (inner == 1) return r * so;
    const int64_t o = r / inner;
    return o * so + (r - o * inner) * si;
}

// A row's pieces of a lane, as they lie in memory; zeros behind its end and of no row.
template <typename T, int CH, bool WHOLE>
__device__ __forceinline__ void row_read(u32x4_t (&raw)[CH], const void *x, int64_t r, int64_t rows, int inner, int64_t so,
                                         int64_t si, int mine, int lanes, int channels)
{
    const T *row = static_cast<const T *>(x) + (r < rows ? norm_at(r, inner, so, si) : 0);
#pragma unroll
    for (int j = 0; j < CH; j++)
        raw[j] = r < rows ? piece_read<T, WHOLE>(row, (mine + j * lanes) * Piece<T>::E, channels) : u32x4_t{0, 0, 0, 0};
}

// MANY: a workgroup's wavefronts share a row, otherwise each has one or several; CH: pieces of a
// lane.  The next row is on its way while this one is summed; weight and bias stay in registers.
template <typename T, bool MANY, int CH, bool WHOLE>
__global__ __launch_bounds__(MANY ? 1024 : 256) void norm_forward(NormArgs A)
{
    typedef Piece<T> P;
    constexpr int E = P::E;
    __shared__ float meet[2][16][1];
    const int lanes = MANY ? (int)blockDim.x : A.lanes;
    const int mine = MANY ? threadIdx.x : threadIdx.x & (lanes - 1);          // the lane's place in its row
    const int per = MANY ? 1 : 256 / lanes;            // rows of a workgroup at a time
    const int own = MANY ? 0 : threadIdx.x / lanes;
    const int64_t step = (int64_t)gridDim.x * per;
    float w[CH][E], b[CH][E];
#pragma unroll
    for (int j = 0; j < CH; j++) {
        param_read<E, WHOLE>(A.w, (mine + j * lanes) * E, A.channels, 1.f, w[j]);
        param_read<E, WHOLE>(A.b, (mine + j * lanes) * E, A.channels, 0.f, b[j]);
    }
    int64_t r = (int64_t)blockIdx.x * per + own;
    u32x4_t raw[CH], next[CH];
    row_read<T, CH, WHOLE>(raw, A.x, r, A.rows, A.inner, A.xs, A.xi, mine, lanes, A.channels);
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < A.rows; r0 += step, r += step) {
        row_read<T, CH, WHOLE>(next, A.x, r + step, A.rows, A.inner, A.xs, A.xi, mine, lanes, A.channels);
        float sum[1] = {0.f};
#pragma unroll
        for (int j = 0; j < CH; j++) {
            float f[E];
            P::open(raw[j], f);
#pragma unroll
            for (int e = 0; e < E; e++) sum[0] += f[e];
        }
        row_sums<MANY, 1>(sum, lanes, meet, 0);
        const float mean = sum[0] * A.part;
        float sq[1] = {0.f};
#pragma unroll
        for (int j = 0; j < CH; j++) {
            const int at = (mine + j * lanes) * E;
            float f[E];
            P::open(raw[j], f);
#pragma unroll
            for (int e = 0; e < E; e++) {
                const float d = at + e < A.channels ? f[e] - mean : 0.f;
                sq[0] = fmaf(d, d, sq[0]);
            }
        }
        row_sums<MANY, 1>(sq, lanes, meet, 1);
        const float rstd = 1.f / sqrtf(fmaf(sq[0], A.part, A.eps));
        if (r < A.rows) {
            if (A.stats && mine == 0) {
                A.stats[2 * r] = mean;
                A.stats[2 * r + 1] = rstd;
            }
            T *y = static_cast<T *>(A.y) + r * A.channels;
#pragma unroll
            for (int j = 0; j < CH; j++) {
                const int at = (mine + j * lanes) * E;
                if (at >= A.channels) continue;
                float f[E];
                P::open(raw[j], f);
#pragma unroll
                for (int e = 0; e < E; e++) f[e] = fmaf((f[e] - mean) * rstd, w[j][e], b[j][e]);
                piece_write<T, WHOLE>(y, at, A.channels, f);
            }
        }
#pragma unroll
        for (int j = 0; j < CH; j++) raw[j] = next[j];
    }
}

template <typename T, bool MANY, int CH, bool WHOLE>
__global__ __launch_bounds__(MANY ? 1024 : 256) void norm_backward(NormArgs A)
{
    typedef Piece<T> P;
    constexpr int E = P::E;
    constexpr bool AHEAD = CH * E <= 8;                  // the next row is on its way
    __shared__ float meet[2][16][2];
    __shared__ __attribute__((aligned(16))) float join[MANY ? 1 : 256 * E];
    const int lanes = MANY ? (int)blockDim.x : A.lanes;
    const int mine = MANY ? threadIdx.x : threadIdx.x & (lanes - 1);
    const int per = MANY ? 1 : 256 / lanes;
    const int own = MANY ? 0 : threadIdx.x / lanes;
    const int64_t step = (int64_t)gridDim.x * per;
    float dw[CH][E], db[CH][E], w[CH][E];
#pragma unroll
    for (int j = 0; j < CH; j++) {
#pragma unroll
        for (int e = 0; e < E; e++) dw[j][e] = db[j][e] = 0.f;
        param_read<E, WHOLE>(A.w, (mine + j * lanes) * E, A.channels, 1.f, w[j]);
    }
    int turn = 0;
    int64_t r = (int64_t)blockIdx.x * per + own;
    u32x4_t rx[CH], rd[CH], nx[CH], nd[CH];
    float mean, rstd, nmean, nrstd;
    auto read = [&](int64_t r, u32x4_t(&rx)[CH], u32x4_t(&rd)[CH], float &mean, float &rstd) {
        row_read<T, CH, WHOLE>(rx, A.x, r, A.rows, A.inner, A.xs, A.xi, mine, lanes, A.channels);
        row_read<T, CH, WHOLE>(rd, A.dy, r, A.rows, A.inner, A.ds, A.di, mine, lanes, A.channels);
        mean = r < A.rows ? *gp(A.stats + 2 * r) : 0.f;
        rstd = r < A.rows ? *gp(A.stats + 2 * r + 1) : 0.f;
    };
    if (AHEAD) read(r, rx, rd, mean, rstd);
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < A.rows; r0 += step, r += step) {
        if (AHEAD) read(r + step, nx, nd, nmean, nrstd);
        else read(r, rx, rd, mean, rstd);
        float sums[2] = {0.f, 0.f};                      // of g and of g xh
#pragma unroll
        for (int j = 0; j < CH; j++) {
            const int at = (mine + j * lanes) * E;
            float f[E], d[E];
            P::open(rx[j], f);
            P::open(rd[j], d);
#pragma unroll
            for (int e = 0; e < E; e++) {
                const float xh = (f[e] - mean) * rstd;
                const float g = at + e < A.channels ? d[e] * w[j][e] : 0.f;
                sums[0] += g;
                sums[1] = at + e < A.channels ? fmaf(g, xh, sums[1]) : sums[1];
                dw[j][e] = fmaf(d[e], xh, dw[j][e]);
                db[j][e] += d[e];
            }
        }
        row_sums<MANY, 2>(sums, lanes, meet, turn);
        turn ^= 1;
        if (r < A.rows) {
            const float mg = sums[0] * A.part, mgx = sums[1] * A.part;
            T *dx = static_cast<T *>(A.dx) + r * A.channels;
#pragma unroll
            for (int j = 0; j < CH; j++) {
                const int at = (mine + j * lanes) * E;
                if (at >= A.channels) continue;
                float f[E], d[E];
                P::open(rx[j], f);
                P::open(rd[j], d);
#pragma unroll
                for (int e = 0; e < E; e++) f[e] = rstd * (fmaf(d[e], w[j][e], -mg) - (f[e] - mean) * rstd * mgx);
                piece_write<T, WHOLE>(dx, at, A.channels, f);
            }
        }
        if (!AHEAD) continue;
#pragma unroll
        for (int j = 0; j < CH; j++) {
            rx[j] = nx[j];
            rd[j] = nd[j];
        }
        mean = nmean;
        rstd = nrstd;
    }
    // one row of sums a workgroup
    for (int which = 0; which < 2; which++) {
        if (!(which ? A.want_b : A.want_w)) continue;
        float *to = A.sums + ((int64_t)blockIdx.x * 2 + which) * A.channels;
#pragma unroll
        for (int j = 0; j < CH; j++) {
            float s[E];
#pragma unroll
            for (int e = 0; e < E; e++) s[e] = which ? db[j][e] : dw[j][e];
            const int at = (mine + j * lanes) * E;
            if (!MANY) {                                 // the rows side by side in the workgroup
                __syncthreads();
#pragma unroll
                for (int e = 0; e < E; e++) join[threadIdx.x * E + e] = s[e];
                __syncthreads();
                if (own == 0)
                    for (int o = 1; o < per; o++)
#pragma unroll
                        for (int e = 0; e < E; e++) s[e] += join[(o * lanes + mine) * E + e];
            }
            if (own == 0)
#pragma unroll
                for (int e = 0; e < E; e++)
                    if (at + e < A.channels) *gp(to + at + e) = s[e];
        }
    }
}

// Adds up the workgroups' rows of sums: 64 columns a workgroup, 16 wavefronts take every 16th
// row each, and the first adds theirs in order.
__global__ __launch_bounds__(1024) void norm_total(const float *sums, int groups, int channels, float *dw, float *db)
{
    __shared__ float meet[16][64];
    const int which = blockIdx.y, wave = threadIdx.x >> 6, l = threadIdx.x & 63, col = blockIdx.x * 64 + l;
    float *to = which ? db : dw;
    if (!to) return;
    float s = 0.f;
    if (col < channels) {
#pragma unroll 8
        for (int g = wave; g < groups; g += 16) s += *gp(sums + ((int64_t)g * 2 + which) * channels + col);
    }
    meet[wave][l] = s;
    __syncthreads();
    if (wave == 0 && col < channels) {
#pragma unroll
        for (int w = 1; w < 16; w++) s += meet[w][l];
        *gp(to + col) = s;
    }
}

}  // namespace emb

using namespace emb;

namespace {

emb_status norm_check(const emb_norm *d)
{
    if (d->dtype != EMB_F32 && d->dtype != EMB_BF16) return fail(EMB_ERR_INVALID_ARG, "layer norm: unknown dtype");
    if (d->channels < 1 || d->inner < 1) return fail(EMB_ERR_INVALID_ARG, "layer norm: channels and inner must be >= 1");
    if (d->channels > kNormChannels) return fail(EMB_ERR_UNSUPPORTED, "layer norm: channels must be <= 16384");
    if (d->rows < 0 || d->rows % d->inner) return fail(EMB_ERR_INVALID_ARG, "layer norm: rows must be a multiple of inner, >= 0");
    if (d->rows > (int64_t(1) << 40)) return fail(EMB_ERR_UNSUPPORTED, "layer norm: rows must be <= 2^40");
    if (d->x_stride < 0 || d->x_inner_stride < 0) return fail(EMB_ERR_INVALID_ARG, "layer norm: strides must be >= 0");
    if (!(d->eps >= 0.f && std::isfinite(d->eps))) return fail(EMB_ERR_INVALID_ARG, "layer norm: eps must be finite and >= 0");
    return EMB_OK;
}

emb_status norm_pointers(const emb_norm *d, const void *y, const void *z)
{
    const size_t el = d->dtype == EMB_BF16 ? 2 : 4;
    if (d->rows && (!d->x || !y || !z)) return fail(EMB_ERR_INVALID_ARG, "layer norm: buffers must be given");
    if (!aligned(d->x, el) || !aligned(y, el) || !aligned(z, el) || !aligned(d->weight, 4) || !aligned(d->bias, 4))
        return fail(EMB_ERR_INVALID_ARG, "layer norm: buffers must be aligned to their elements");
    return EMB_OK;
}

// A row of up to 1024 channels is one wavefront's or a part's of one, a longer one is a workgroup's
// with a wavefront for every 1024: 16 channels a lane at most, the most whose sums, weights and
// pieces fit in the registers.  8 a lane and twice the wavefronts was slower where that makes one
// wavefront two (60000 rows of 768 in bf16, backward: 83 us, here 56; 30000 of 1024: 49 and 39)
// and no faster above (8191 of 5000 in fp32: 105 and 108).
struct NormPlan {
    int waves, pieces, lanes;
    int64_t at_once, groups;             // rows of a workgroup at a time; workgroups that have one
};

NormPlan norm_plan(const emb_norm *d)
{
    NormPlan p{};
    const int E = d->dtype == EMB_BF16 ? 8 : 4;
    const int n = (d->channels + E - 1) / E;
    p.lanes = 1;
    while (p.lanes < 64 && p.lanes < n) p.lanes *= 2;
    p.waves = (d->channels + 1023) / 1024;
    p.pieces = p.waves > 1 || n > 128 ? 16 / E : n > 64 ? 2 : 1;
    p.at_once = p.waves == 1 ? 256 / p.lanes : 1;
    p.groups = (d->rows + p.at_once - 1) / p.at_once;
    return p;
}

// Workgroups.  The forward takes what keeps the card busy to the end (140771 rows of 512 bf16: 1024
// workgroups 73 us, 8192 55, one a set of rows 62; 4000 of 16384: 1024 of 16 wavefronts 53 us,
// 4096 60).  Each of the backward writes sums of its own, which norm_total reads again: no more
// than run at the same time (140771 x 512: 512 109 us, 768 88, 1024 88, 1536 108; 30000 x 1024: 39 at
// 768, 44 at 1024; 8191 x 5000 fp32, 5 wavefronts: 256 114, 512 108, 1024 122; 4000 x 16384: 256 100, 512 123).
int64_t norm_groups(const NormPlan &p, bool backward)
{
    const int64_t most = backward ? p.waves == 1 ? 768 : 256 * (p.waves < 10 ? 10 / p.waves : 1)
                                  : p.waves == 1 ? 8192 : 16384 / p.waves;
    return p.groups < most ? p.groups : most;
}

NormArgs norm_args(const emb_norm *d, const NormPlan &p)
{
    NormArgs A{};
    A.x = d->x;
    A.xs = d->x_stride;
    A.xi = d->x_inner_stride;
    A.w = d->weight;
    A.b = d->bias;
    A.rows = d->rows;
    A.inner = d->inner;
    A.channels = d->channels;
    A.lanes = p.lanes;
    A.eps = d->eps;
    A.part = (float)(1.0 / d->channels);
    return A;
}

template <typename T, bool MANY, int CH>
void norm_launch_one(const NormArgs &A, int waves, int64_t groups, bool backward, hipStream_t st)
{
    const dim3 grid((unsigned)groups), block(MANY ? 64 * waves : 256);
    const bool whole = A.channels % Piece<T>::E == 0;
    const auto kernel = backward ? whole ? norm_backward<T, MANY, CH, true> : norm_backward<T, MANY, CH, false>
                                 : whole ? norm_forward<T, MANY, CH, true> : norm_forward<T, MANY, CH, false>;
    hipLaunchKernelGGL(kernel, grid, block, 0, st, A);
}

template <typename T>
void norm_launch(const NormArgs &A, const NormPlan &p, int64_t groups, bool backward, hipStream_t st)
{
    constexpr int most = 16 / Piece<T>::E;
    if (p.waves > 1) norm_launch_one<T, true, most>(A, p.waves, groups, backward, st);
    else if (p.pieces == 1) norm_launch_one<T, false, 1>(A, 1, groups, backward, st);
    else if (p.pieces == 2) norm_launch_one<T, false, 2>(A, 1, groups, backward, st);
    else norm_launch_one<T, false, most>(A, 1, groups, backward, st);
}

emb_status norm_launched()
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(EMB_ERR_HIP, std::string("layer norm launch: ") + hipGetErrorString(e));
    return EMB_OK;
}

size_t norm_workspace(const emb_norm *d, const NormPlan &p)
{
    return (size_t)norm_groups(p, true) * 2 * d->channels * 4;
}

}  // namespace

extern "C" emb_status emb_norm_query(const emb_norm *d, size_t *backward_bytes)
{
    if (!d) return fail(EMB_ERR_INVALID_ARG, "layer norm descriptor is NULL");
    const emb_status s = norm_check(d);
    if (s != EMB_OK) return s;
    if (!backward_bytes) return fail(EMB_ERR_INVALID_ARG, "layer norm: output pointers must be given");
    *backward_bytes = norm_workspace(d, norm_plan(d));
    return EMB_OK;
}

extern "C" emb_status emb_norm_forward(const emb_norm *d, void *y, float *stats, void *stream)
{
    if (!d) return fail(EMB_ERR_INVALID_ARG, "layer norm descriptor is NULL");
    emb_status s = norm_check(d);
    if (s == EMB_OK) s = norm_pointers(d, y, y);
    if (s != EMB_OK) return s;
    if (!aligned(stats, 4)) return fail(EMB_ERR_INVALID_ARG, "layer norm: stats must be 4-byte aligned");
    if (!d->rows) return EMB_OK;
    const NormPlan p = norm_plan(d);
    NormArgs A = norm_args(d, p);
    A.y = y;
    A.stats = stats;
    const int64_t groups = norm_groups(p, false);
    if (d->dtype == EMB_BF16) norm_launch<uint16_t>(A, p, groups, false, static_cast<hipStream_t>(stream));
    else norm_launch<float>(A, p, groups, false, static_cast<hipStream_t>(stream));
    return norm_launched();
}

extern "C" emb_status emb_norm_backward(const emb_norm *d, const float *stats, const void *dy, int64_t dy_stride,
                                        int64_t dy_inner_stride, void *dx, float *dweight, float *dbias, void *workspace,
                                        size_t workspace_bytes, void *stream)
{
    if (!d) return fail(EMB_ERR_INVALID_ARG, "layer norm descriptor is NULL");
    emb_status s = norm_check(d);
    if (s == EMB_OK) s = norm_pointers(d, dy, dx);
    if (s != EMB_OK) return s;
    if (dy_stride < 0 || dy_inner_stride < 0) return fail(EMB_ERR_INVALID_ARG, "layer norm: strides must be >= 0");
    if (d->rows && !stats) return fail(EMB_ERR_INVALID_ARG, "layer norm: stats must be given");
    if (!aligned(stats, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return fail(EMB_ERR_INVALID_ARG, "layer norm: buffers must be aligned to their elements");
    const NormPlan p = norm_plan(d);
    const bool sums = dweight || dbias;
    if (sums && d->rows && (workspace_bytes < norm_workspace(d, p) || !workspace || !aligned(workspace, 4)))
        return fail(EMB_ERR_WORKSPACE, "layer norm: the workspace is smaller than the query returned, or not 4-byte aligned");
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t groups = norm_groups(p, true);
    if (groups) {
        NormArgs A = norm_args(d, p);
        A.stats = const_cast<float *>(stats);
        A.dy = dy;
        A.ds = dy_stride;
        A.di = dy_inner_stride;
        A.dx = dx;
        A.sums = static_cast<float *>(workspace);
        A.want_w = dweight != nullptr;
        A.want_b = dbias != nullptr;
        if (d->dtype == EMB_BF16) norm_launch<uint16_t>(A, p, groups, true, st);
        else norm_launch<float>(A, p, groups, true, st);
    }
    if (sums)
        hipLaunchKernelGGL(norm_total, dim3((unsigned)((d->channels + 63) / 64), 2), dim3(1024), 0, st,
                           static_cast<const float *>(workspace), (int)groups, d->channels, dweight, dbias);
    return norm_launched();
}
