// recurrence.hip -- the gated linear recurrence over jagged sequences,
//   a_t = sigmoid(gate_t),  h_t = a_t h_(t-1) + (1 - a_t) x_t  in every channel,
// its backward pass and its one-step form.
#include <string>

#include "sequence.h"

namespace emb {

constexpr int kScanSteps = 16;   // consecutive steps a wavefront of the forward holds in registers
constexpr int kBackSteps = 8;    // ... of the backward, which holds twice as much per step
constexpr int kChunk = 512;      // rows per chunk of a split scan
constexpr int kSaved = 8;        // the forward saves the state before every kSaved steps

struct ScanArgs {
    const void *x, *gate;        // [n, channels], rows xs / gs elements apart
    int64_t xs, gs;
    const int32_t *off;          // [samples + 1]
    const uint8_t *mask;         // [n] or NULL
    const float *state;          // [samples, channels] or NULL
    void *y;                     // [n, channels]
    float *last;                 // [samples, channels]
    float *ckpt;                 // state before each group of kSaved steps, or NULL
    const void *dy;              // backward
    const float *dlast;
    void *dx, *dgate;
    float *dstate;
    float *sum_a, *sum_h;        // [tiles, channels]: what a chunk does to the state it is given
    int64_t n, tiles;
    int32_t samples, channels;
    int32_t chunk;               // samples are cut into chunks of kChunk rows
};

// sigmoid(g) and sigmoid(-g) = 1 - sigmoid(g), the small one without cancellation:
// e = exp(-|g|), the larger is 1 / (1 + e), the smaller e / (1 + e).
__device__ __forceinline__ void sigmoid_pair(float g, float &a, float &na)
{
    const float e = exp2_fast(-fabsf(g) * kLog2e);
    const float big = __builtin_amdgcn_rcpf(1.f + e), small = e * big;
    a = g >= 0.f ? big : small;
    na = g >= 0.f ? small : big;
}

// VEC neighbouring channels of one row as they lie in memory, and as floats
template <typename T, int VEC>
struct Chan;
template <>
struct Chan<float, 1> {
    typedef float Raw;
    static __device__ __forceinline__ void open(Raw r, float *v) { v[0] = r; }
    static __device__ __forceinline__ Raw pack(const float *v) { return v[0]; }
};
template <>
struct Chan<float, 2> {
    typedef float2 Raw;
    static __device__ __forceinline__ void open(Raw r, float *v)
    {
        v[0] = r.x;
        v[1] = r.y;
    }
    static __device__ __forceinline__ Raw pack(const float *v) { return make_float2(v[0], v[1]); }
};
template <>
struct Chan<uint16_t, 1> {
    typedef uint16_t Raw;
    static __device__ __forceinline__ void open(Raw r, float *v) { v[0] = bf16_lo(r); }
    static __device__ __forceinline__ Raw pack(const float *v) { return bf16_rne(v[0]); }
};
template <>
struct Chan<uint16_t, 2> {
    typedef uint32_t Raw;
    static __device__ __forceinline__ void open(Raw r, float *v)
    {
        v[0] = bf16_lo(r);
        v[1] = bf16_hi(r);
    }
    static __device__ __forceinline__ Raw pack(const float *v) { return bf16x2_rne(v[0], v[1]); }
};

// row (uniform) and channel c (per lane) of a tensor
template <typename R, typename T>
__device__ __forceinline__ R row_load(const T *p, int64_t row, int64_t stride, uint32_t c)
{
    return *gp(reinterpret_cast<const R *>(p + row * stride + c));
}
template <typename R, typename T>
__device__ __forceinline__ void row_store(T *p, int64_t row, int64_t stride, uint32_t c, R v)
{
    *gp(reinterpret_cast<R *>(p + row * stride + c)) = v;
}

// Which rows a workgroup walks: one sample, or one chunk of one.
struct ScanSpan {
    int64_t begin, end;      // rows
    int64_t first;           // first row of the sample
    int64_t tile, tile0;     // chunk number, that of the sample's first chunk
    int64_t chunks;          // of the sample
    int seg;
};

__device__ __forceinline__ bool scan_span(const ScanArgs &A, int64_t block, ScanSpan &s)
{
    s.tile = block;
    if (A.chunk == 0) {
        s.seg = (int)block;
        s.tile0 = block;
        s.chunks = 1;
        s.first = s.begin = seg_edge(A.off, A.samples, (int)A.n, s.seg);
        s.end = seg_edge(A.off, A.samples, (int)A.n, s.seg + 1);
        return true;
    }
    const SegTile t = seg_find<kChunk>(A.off, (int)A.n, nullptr, 0, A.samples, 1, (int)block);
    s.seg = t.seg;
    s.first = t.base;
    s.tile0 = t.base / kChunk + t.seg;
    s.chunks = (t.rows + kChunk - 1) / kChunk;
    s.begin = t.base + t.row0;
    s.end = t.row0 + kChunk < t.rows ? s.begin + kChunk : t.base + t.rows;
    // an empty sample keeps its first chunk: it hands the state through
    return t.row0 < t.rows || (t.rows == 0 && t.row0 == 0);
}

// The saved state of the group of kSaved rows that begins at `row`
__device__ __forceinline__ int64_t saved_row(const ScanSpan &s, int64_t row)
{
    return s.first / kSaved + s.seg + (row - s.first) / kSaved;
}

enum { kScanWhole = 0, kScanSum = 1, kScanApply = 2 };

// What the pairs (A, H) of the sample's chunks before this one (after it, in the
// backward) make of the state v: each wavefront folds its share of the pairs, and the
// W results meet in LDS.
template <int VEC, int W, bool REVERSE>
__device__ __forceinline__ void chunk_state(const ScanArgs &A, const ScanSpan &s, int w, uint32_t c,
                                            float (&pa)[W][64 * VEC], float (&ph)[W][64 * VEC], float *v)
{
    const int64_t here = s.tile - s.tile0, n = REVERSE ? s.chunks - 1 - here : here, C = A.channels;
    const int64_t i0 = n * w / W, i1 = n * (w + 1) / W;
    const int lane = lane_id();
    float a[VEC], h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; e++) {
        a[e] = 1.f;
        h[e] = 0.f;
    }
    constexpr int kAhead = 8;    // pairs loaded before the first is needed
    for (int64_t i = i0; i < i1; i += kAhead) {
        float ra[kAhead][VEC], rh[kAhead][VEC];
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            const int64_t k = i + j < i1 ? i + j : i1 - 1;
            const int64_t t = s.tile0 + (REVERSE ? s.chunks - 1 - k : k);
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                ra[j][e] = row_load<float>(A.sum_a, t, C, c + e);
                rh[j][e] = row_load<float>(A.sum_h, t, C, c + e);
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; j++)
            if (i + j < i1)
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    h[e] = fmaf(ra[j][e], h[e], rh[j][e]);
                    a[e] *= ra[j][e];
                }
    }
#pragma unroll
    for (int e = 0; e < VEC; e++) {
        pa[w][lane * VEC + e] = a[e];
        ph[w][lane * VEC + e] = h[e];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < W; u++)
#pragma unroll
        for (int e = 0; e < VEC; e++) v[e] = fmaf(pa[u][lane * VEC + e], v[e], ph[u][lane * VEC + e]);
    __syncthreads();
}

// W wavefronts walk a sample (or chunk) in blocks of W * kScanSteps rows: each
// loads its own kScanSteps rows of 64 * VEC channels, scans them from a zero state
// into (A, H) with h_out = A h_in + H, the W pairs meet in LDS, and each wavefront
// applies its rows from the state that the pairs before it give.  One pass over the
// data; the state stays in fp32 registers.  Rows past the end and masked ones load
// some other row of the sample and count as a = 1, x = 0; the next block's rows are
// loaded before this block's arithmetic.
template <typename T, int VEC, int W, int PHASE>
__global__ __launch_bounds__(64 * W, W == 8 ? 4 : 1) void scan_forward(ScanArgs A)
{
    typedef Chan<T, VEC> CH;
    typedef typename CH::Raw Raw;
    __shared__ float pa[2][W][64 * VEC], ph[2][W][64 * VEC];
    const int lane = lane_id(), w = uniform((int)(threadIdx.x >> 6));
    const uint32_t cw = (blockIdx.y * 64 + lane) * VEC;
    const bool live = cw < (uint32_t)A.channels;
    const uint32_t c = live ? cw : 0;      // lanes past the last channel repeat the first
    const int64_t C = A.channels;
    ScanSpan s;
    if (!scan_span(A, blockIdx.x, s)) return;
    const T *x = static_cast<const T *>(A.x), *gate = static_cast<const T *>(A.gate);
    T *y = static_cast<T *>(A.y);
    if (s.seg == 0 || s.seg == A.samples + 1) {
        const float z[VEC] = {};
        if (PHASE != kScanSum && live)
            for (int64_t t = s.begin + w; t < s.end; t += W) row_store(y, t, C, c, CH::pack(z));
        return;
    }
    float h[VEC], ta[VEC];
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        h[v] = PHASE != kScanSum && A.state ? A.state[(int64_t)(s.seg - 1) * C + c + v] : 0.f;
        ta[v] = 1.f;
    }
    if (PHASE == kScanApply) chunk_state<VEC, W, false>(A, s, w, c, pa[0], ph[0], h);

    Raw xn[kScanSteps], gn[kScanSteps];
    uint32_t keep = 0;
    auto load = [&](int64_t t0) {
        const int64_t mine = t0 + w * kScanSteps;
        keep = lane < kScanSteps && mine + lane < s.end ? (A.mask ? *gp(A.mask + mine + lane) : 1) : 0;
#pragma unroll
        for (int i = 0; i < kScanSteps; i++) {
            const int64_t row = mine + i < s.end ? mine + i : s.end - 1;
            xn[i] = row_load<Raw>(x, row, A.xs, c);
            gn[i] = row_load<Raw>(gate, row, A.gs, c);
        }
    };
    if (s.begin < s.end) load(s.begin);
    int buf = 0;
    for (int64_t t0 = s.begin; t0 < s.end; t0 += W * kScanSteps, buf ^= 1) {
        const int64_t mine = t0 + w * kScanSteps;
        const uint32_t bits = (uint32_t)__ballot(keep != 0);
        float xs[kScanSteps][VEC], as[kScanSteps][VEC], la[VEC], lh[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            la[v] = 1.f;
            lh[v] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kScanSteps; i++) {
            const bool on = bits >> i & 1;
            CH::open(xn[i], xs[i]);
            CH::open(gn[i], as[i]);
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                float na;
                sigmoid_pair(on ? as[i][v] : INFINITY, as[i][v], na);
                xs[i][v] = na * (on ? xs[i][v] : 0.f);
                lh[v] = fmaf(as[i][v], lh[v], xs[i][v]);
                la[v] *= as[i][v];
            }
        }
        if (t0 + W * kScanSteps < s.end) load(t0 + W * kScanSteps);
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            pa[buf][w][lane * VEC + v] = la[v];
            ph[buf][w][lane * VEC + v] = lh[v];
        }
        __syncthreads();
        float in[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) in[v] = h[v];
#pragma unroll
        for (int u = 0; u < W; u++)
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                if (u == w) in[v] = h[v];
                const float ua = pa[buf][u][lane * VEC + v];
                h[v] = fmaf(ua, h[v], ph[buf][u][lane * VEC + v]);
                if (PHASE == kScanSum) ta[v] *= ua;
            }
        if (PHASE == kScanSum) continue;
#pragma unroll
        for (int i = 0; i < kScanSteps; i++) {
            if (A.ckpt && i % kSaved == 0 && live && mine + i < s.end)
#pragma unroll
                for (int v = 0; v < VEC; v++) row_store(A.ckpt, saved_row(s, mine + i), C, c + v, in[v]);
#pragma unroll
            for (int v = 0; v < VEC; v++) in[v] = fmaf(as[i][v], in[v], xs[i][v]);
            if (live && mine + i < s.end) row_store(y, mine + i, C, c, CH::pack(in));
        }
    }
    if (!live || w != 0) return;
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        if (PHASE == kScanWhole || (PHASE == kScanApply && s.tile - s.tile0 >= s.chunks - 1))
            A.last[(int64_t)(s.seg - 1) * C + c + v] = h[v];
        if (PHASE == kScanSum) {
            row_store(A.sum_a, s.tile, C, c + v, ta[v]);
            row_store(A.sum_h, s.tile, C, c + v, h[v]);
        }
    }
}

// The backward pass walks the same blocks from the last to the first.  With
// u_t = a_t g_t the carried quantity, g_t = dy_t + u_(t+1) is the gradient of h_t,
// again a linear recurrence.  The states h_(t-1) that dgate needs are scanned again
// from the saved state before each group of kSaved rows: an eighth of the states in
// fp32 is a quarter of what all of them in bf16 would cost, and exact.
template <typename T, int VEC, int W, int PHASE>
__global__ __launch_bounds__(64 * W, W == 8 ? 4 : 1) void scan_backward(ScanArgs A)
{
    typedef Chan<T, VEC> CH;
    typedef typename CH::Raw Raw;
    __shared__ float pa[2][W][64 * VEC], ph[2][W][64 * VEC];
    const int lane = lane_id(), w = uniform((int)(threadIdx.x >> 6));
    const uint32_t cw = (blockIdx.y * 64 + lane) * VEC;
    const bool live = cw < (uint32_t)A.channels;
    const uint32_t c = live ? cw : 0;
    const int64_t C = A.channels;
    ScanSpan s;
    if (!scan_span(A, blockIdx.x, s)) return;
    const T *x = static_cast<const T *>(A.x), *gate = static_cast<const T *>(A.gate);
    const T *dy = static_cast<const T *>(A.dy);
    T *dx = static_cast<T *>(A.dx), *dgate = static_cast<T *>(A.dgate);
    if (s.seg == 0 || s.seg == A.samples + 1) {
        const float z[VEC] = {};
        if (PHASE != kScanSum && live)
            for (int64_t t = s.begin + w; t < s.end; t += W) {
                row_store(dx, t, C, c, CH::pack(z));
                row_store(dgate, t, C, c, CH::pack(z));
            }
        return;
    }
    float u[VEC], ta[VEC];
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        u[v] = PHASE != kScanSum && A.dlast ? A.dlast[(int64_t)(s.seg - 1) * C + c + v] : 0.f;
        ta[v] = 1.f;
    }
    if (PHASE == kScanApply) chunk_state<VEC, W, true>(A, s, w, c, pa[0], ph[0], u);

    constexpr int kRows = W * kBackSteps;
    const int64_t blocks = s.end > s.begin ? (s.end - s.begin + kRows - 1) / kRows : 0;
    Raw xn[kBackSteps], gn[kBackSteps], dn[kBackSteps];
    float hn[VEC];
    uint32_t keep = 0;
    auto load = [&](int64_t b) {
        const int64_t mine = s.begin + b * kRows + w * kBackSteps;
        keep = lane < kBackSteps && mine + lane < s.end ? (A.mask ? *gp(A.mask + mine + lane) : 1) : 0;
#pragma unroll
        for (int i = 0; i < kBackSteps; i++) {
            const int64_t row = mine + i < s.end ? mine + i : s.end - 1;
            if (PHASE != kScanSum) xn[i] = row_load<Raw>(x, row, A.xs, c);
            gn[i] = row_load<Raw>(gate, row, A.gs, c);
            dn[i] = row_load<Raw>(dy, row, C, c);
        }
#pragma unroll
        for (int v = 0; v < VEC; v++)
            if (PHASE != kScanSum)
                hn[v] = row_load<float>(A.ckpt, saved_row(s, mine < s.end ? mine : s.begin), C, c + v);
    };
    if (blocks) load(blocks - 1);
    int buf = 0;
    for (int64_t b = blocks - 1; b >= 0; b--, buf ^= 1) {
        const int64_t mine = s.begin + b * kRows + w * kBackSteps;
        const uint32_t bits = (uint32_t)__ballot(keep != 0);
        float xs[kBackSteps][VEC], as[kBackSteps][VEC], na[kBackSteps][VEC], ds[kBackSteps][VEC], hin[VEC];
        float la[VEC], lu[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            la[v] = 1.f;
            lu[v] = 0.f;
            hin[v] = PHASE != kScanSum ? hn[v] : 0.f;
        }
#pragma unroll
        for (int i = kBackSteps - 1; i >= 0; i--) {
            const bool on = bits >> i & 1, in = mine + i < s.end;
            CH::open(gn[i], as[i]);
            CH::open(dn[i], ds[i]);
            if (PHASE != kScanSum) CH::open(xn[i], xs[i]);
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                sigmoid_pair(on ? as[i][v] : INFINITY, as[i][v], na[i][v]);
                ds[i][v] = in ? ds[i][v] : 0.f;
                if (PHASE != kScanSum) xs[i][v] = on ? xs[i][v] : 0.f;
                lu[v] = as[i][v] * (ds[i][v] + lu[v]);
                la[v] *= as[i][v];
            }
        }
        if (b > 0) load(b - 1);
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            pa[buf][w][lane * VEC + v] = la[v];
            ph[buf][w][lane * VEC + v] = lu[v];
        }
        __syncthreads();
        float in[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) in[v] = u[v];
#pragma unroll
        for (int p = W - 1; p >= 0; p--)
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                if (p == w) in[v] = u[v];
                const float pv = pa[buf][p][lane * VEC + v];
                u[v] = fmaf(pv, u[v], ph[buf][p][lane * VEC + v]);
                if (PHASE == kScanSum) ta[v] *= pv;
            }
        if (PHASE == kScanSum) continue;
        // forward again: xs becomes h_(t-1) - x_t, what dgate multiplies
#pragma unroll
        for (int i = 0; i < kBackSteps; i++)
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                const float before = hin[v];
                hin[v] = fmaf(as[i][v], before, na[i][v] * xs[i][v]);
                xs[i][v] = before - xs[i][v];
            }
#pragma unroll
        for (int i = kBackSteps - 1; i >= 0; i--) {
            float gx[VEC], gg[VEC];
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                const float g = ds[i][v] + in[v];
                in[v] = as[i][v] * g;
                gx[v] = na[i][v] * g;                        // a masked row has na = 0
                gg[v] = as[i][v] * xs[i][v] * gx[v];
            }
            if (live && mine + i < s.end) {
                row_store(dx, mine + i, C, c, CH::pack(gx));
                row_store(dgate, mine + i, C, c, CH::pack(gg));
            }
        }
    }
    if (!live || w != 0) return;
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        if (A.dstate && (PHASE == kScanWhole || (PHASE == kScanApply && s.tile == s.tile0)))
            A.dstate[(int64_t)(s.seg - 1) * C + c + v] = u[v];
        if (PHASE == kScanSum) {
            row_store(A.sum_a, s.tile, C, c + v, ta[v]);
            row_store(A.sum_h, s.tile, C, c + v, u[v]);
        }
    }
}

template <typename T, int VEC>
__global__ __launch_bounds__(256) void scan_step(const T *x, const T *gate, int64_t xs, int64_t gs,
                                                 float *state, T *y, int64_t rows, int64_t C)
{
    const int64_t per = (C + VEC - 1) / VEC;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * per) return;
    const int64_t b = i / per, c = (i - b * per) * VEC;
    typedef Chan<T, VEC> CH;
    typedef Chan<float, VEC> CF;
    float xv[VEC], gv[VEC], h[VEC];
    CH::open(*gp(reinterpret_cast<const typename CH::Raw *>(x + b * xs + c)), xv);
    CH::open(*gp(reinterpret_cast<const typename CH::Raw *>(gate + b * gs + c)), gv);
    CF::open(*gp(reinterpret_cast<const typename CF::Raw *>(state + b * C + c)), h);
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        float a, na;
        sigmoid_pair(gv[v], a, na);
        h[v] = fmaf(a, h[v], na * xv[v]);
    }
    *gp(reinterpret_cast<typename CF::Raw *>(state + b * C + c)) = CF::pack(h);
    *gp(reinterpret_cast<typename CH::Raw *>(y + b * C + c)) = CH::pack(h);
}

}  // namespace emb

using namespace emb;

namespace {

struct ScanPlan {
    int waves, vec;
    int32_t chunk;               // cut samples into chunks
    int64_t tiles, ckpt_rows;
};

// One workgroup walks a whole sample when the samples and channel blocks alone fill
// the chip; otherwise samples are cut into chunks.
ScanPlan scan_plan(const emb_recurrence *r)
{
    ScanPlan p{};
    const int64_t mean = r->samples ? r->n / r->samples : 0;
    p.waves = mean <= 32 ? 1 : 8;
    const int64_t per = r->dtype == EMB_BF16 ? 128 : 64;
    const int64_t blocks = (r->channels + per - 1) / per;
    p.chunk = 0;
    p.tiles = r->samples + 2;
    if (r->samples * blocks < 512 && mean >= 1024) {
        p.chunk = 1;
        p.tiles = seg_tiles(r->n, r->samples, 1, kChunk);
    }
    p.ckpt_rows = seg_tiles(r->n, r->samples, 1, kSaved);
    return p;
}

emb_status scan_check(const emb_recurrence *r)
{
    if (!r) return fail(EMB_ERR_INVALID_ARG, "recurrence descriptor is NULL");
    if (r->dtype != EMB_F32 && r->dtype != EMB_BF16) return fail(EMB_ERR_INVALID_ARG, "recurrence: unknown dtype");
    if (r->samples < 0 || r->n < 0) return fail(EMB_ERR_INVALID_ARG, "recurrence: samples and n must be >= 0");
    if (r->channels <= 0) return fail(EMB_ERR_INVALID_ARG, "recurrence: channels must be >= 1");
    if (r->channels > (1 << 20)) return fail(EMB_ERR_UNSUPPORTED, "recurrence: channels must be <= 2^20");
    if (r->n > kRowsMost || r->samples > (1 << 30))
        return fail(EMB_ERR_UNSUPPORTED, "recurrence: n must be <= 2^31 - 65536 and samples <= 2^30");
    if (r->x_stride < 0 || r->gate_stride < 0)
        return fail(EMB_ERR_INVALID_ARG, "recurrence: row strides must be >= 0");
    return EMB_OK;
}

emb_status scan_pointers(const emb_recurrence *r)
{
    const size_t el = r->dtype == EMB_BF16 ? 2 : 4;
    if (!r->offsets || !aligned(r->offsets, 4)) return fail(EMB_ERR_INVALID_ARG, "recurrence: offsets must be given");
    if (r->n && (!r->x || !r->gate)) return fail(EMB_ERR_INVALID_ARG, "recurrence: x and gate must be given");
    if (!aligned(r->x, el) || !aligned(r->gate, el))
        return fail(EMB_ERR_INVALID_ARG, "recurrence: x and gate must be aligned to their elements");
    if (!aligned(r->state, 4)) return fail(EMB_ERR_INVALID_ARG, "recurrence: state must be 4-byte aligned");
    return EMB_OK;
}

size_t pad256(size_t x) { return (x + 255) & ~size_t(255); }

size_t scan_workspace(const emb_recurrence *r, const ScanPlan &p)
{
    return p.chunk ? 2 * pad256((size_t)p.tiles * r->channels * 4) : 0;
}

// channels in pairs: an even count, and every row aligned to a pair
bool pairs_ok(const emb_recurrence *r, std::initializer_list<const void *> same)
{
    const size_t el = r->dtype == EMB_BF16 ? 2 : 4;
    if (r->channels % 2 || r->x_stride % 2 || r->gate_stride % 2) return false;
    if (!aligned(r->x, 2 * el) || !aligned(r->gate, 2 * el)) return false;
    for (const void *p : same)
        if (!aligned(p, 2 * el)) return false;
    return true;
}

template <typename T, int VEC, int W>
emb_status scan_launch_w(const ScanArgs &A, bool backward, hipStream_t st)
{
    const int64_t blocks = (A.channels + 64 * VEC - 1) / (64 * VEC);
    const dim3 grid((unsigned)A.tiles, (unsigned)blocks), block(64 * W);
    if (A.chunk == 0) {
        if (backward) hipLaunchKernelGGL((scan_backward<T, VEC, W, kScanWhole>), grid, block, 0, st, A);
        else hipLaunchKernelGGL((scan_forward<T, VEC, W, kScanWhole>), grid, block, 0, st, A);
    } else if (backward) {
        hipLaunchKernelGGL((scan_backward<T, VEC, W, kScanSum>), grid, block, 0, st, A);
        hipLaunchKernelGGL((scan_backward<T, VEC, W, kScanApply>), grid, block, 0, st, A);
    } else {
        hipLaunchKernelGGL((scan_forward<T, VEC, W, kScanSum>), grid, block, 0, st, A);
        hipLaunchKernelGGL((scan_forward<T, VEC, W, kScanApply>), grid, block, 0, st, A);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(EMB_ERR_HIP, std::string("recurrence launch: ") + hipGetErrorString(e));
    return EMB_OK;
}

template <typename T, int VEC>
emb_status scan_launch_v(const ScanArgs &A, int waves, bool backward, hipStream_t st)
{
    return waves == 1 ? scan_launch_w<T, VEC, 1>(A, backward, st) : scan_launch_w<T, VEC, 8>(A, backward, st);
}

emb_status scan_launch(const emb_recurrence *r, const ScanArgs &A, int waves, bool pairs, bool backward,
                       void *stream)
{
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (r->dtype == EMB_BF16)
        return pairs ? scan_launch_v<uint16_t, 2>(A, waves, backward, st)
                     : scan_launch_v<uint16_t, 1>(A, waves, backward, st);
    return scan_launch_v<float, 1>(A, waves, backward, st);
}

ScanArgs scan_args(const emb_recurrence *r, const ScanPlan &p, void *ws)
{
    ScanArgs A{};
    A.x = r->x;
    A.gate = r->gate;
    A.xs = r->x_stride;
    A.gs = r->gate_stride;
    A.off = r->offsets;
    A.mask = r->mask;
    A.state = r->state;
    A.n = r->n;
    A.samples = r->samples;
    A.channels = r->channels;
    A.chunk = p.chunk;
    A.tiles = p.tiles;
    if (p.chunk) {
        const size_t part = pad256((size_t)p.tiles * r->channels * 4);
        A.sum_a = reinterpret_cast<float *>(ws);
        A.sum_h = reinterpret_cast<float *>(static_cast<char *>(ws) + part);
    }
    return A;
}

}  // namespace

extern "C" emb_status emb_recurrence_query(const emb_recurrence *r, int64_t *saved_rows, size_t *workspace_bytes)
{
    const emb_status s = scan_check(r);
    if (s != EMB_OK) return s;
    if (!saved_rows || !workspace_bytes) return fail(EMB_ERR_INVALID_ARG, "recurrence: output pointers must be given");
    const ScanPlan p = scan_plan(r);
    *saved_rows = p.ckpt_rows;
    *workspace_bytes = scan_workspace(r, p);
    return EMB_OK;
}

extern "C" emb_status emb_recurrence_forward(const emb_recurrence *r, void *y, float *last, float *saved,
                                             void *workspace, size_t workspace_bytes, void *stream)
{
    emb_status s = scan_check(r);
    if (s == EMB_OK) s = scan_pointers(r);
    if (s != EMB_OK) return s;
    const size_t el = r->dtype == EMB_BF16 ? 2 : 4;
    if ((r->n && !y) || (r->samples && !last) || !aligned(y, el) || !aligned(last, 4) || !aligned(saved, 4))
        return fail(EMB_ERR_INVALID_ARG, "recurrence: y and last must be given and aligned");
    const ScanPlan p = scan_plan(r);
    if (workspace_bytes < scan_workspace(r, p) || (scan_workspace(r, p) && !aligned(workspace, 256)))
        return fail(EMB_ERR_WORKSPACE, "recurrence: the workspace is smaller than the query returned, or not 256-byte aligned");
    if (p.chunk && !workspace) return fail(EMB_ERR_WORKSPACE, "recurrence: workspace is NULL");
    ScanArgs A = scan_args(r, p, workspace);
    A.y = y;
    A.last = last;
    A.ckpt = saved;
    return scan_launch(r, A, p.waves, pairs_ok(r, {y}), false, stream);
}

extern "C" emb_status emb_recurrence_backward(const emb_recurrence *r, const float *saved, const void *dy,
                                              const float *dlast, void *dx, void *dgate, float *dstate,
                                              void *workspace, size_t workspace_bytes, void *stream)
{
    emb_status s = scan_check(r);
    if (s == EMB_OK) s = scan_pointers(r);
    if (s != EMB_OK) return s;
    const size_t el = r->dtype == EMB_BF16 ? 2 : 4;
    if (r->n && (!dy || !dx || !dgate || !saved))
        return fail(EMB_ERR_INVALID_ARG, "recurrence: saved, dy, dx and dgate must be given");
    if (!aligned(dy, el) || !aligned(dx, el) || !aligned(dgate, el) || !aligned(saved, 4) || !aligned(dlast, 4) ||
        !aligned(dstate, 4))
        return fail(EMB_ERR_INVALID_ARG, "recurrence: buffers must be aligned to their elements");
    const ScanPlan p = scan_plan(r);
    if (workspace_bytes < scan_workspace(r, p) || (scan_workspace(r, p) && !aligned(workspace, 256)))
        return fail(EMB_ERR_WORKSPACE, "recurrence: the workspace is smaller than the query returned, or not 256-byte aligned");
    if (p.chunk && !workspace) return fail(EMB_ERR_WORKSPACE, "recurrence: workspace is NULL");
    ScanArgs A = scan_args(r, p, workspace);
    A.dy = dy;
    A.dlast = dlast;
    A.dx = dx;
    A.dgate = dgate;
    A.dstate = dstate;
    A.ckpt = const_cast<float *>(saved);
    return scan_launch(r, A, p.waves, pairs_ok(r, {dy, dx, dgate}), true, stream);
}

extern "C" emb_status emb_recurrence_step(int32_t dtype, int64_t rows, int32_t channels, const void *x,
                                          int64_t x_stride, const void *gate, int64_t gate_stride,
                                          float *state, void *y, void *stream)
{
    emb_recurrence r{};
    r.dtype = dtype;
    r.channels = channels;
    r.n = rows;
    r.x_stride = x_stride;
    r.gate_stride = gate_stride;
    r.x = x;
    r.gate = gate;
    const emb_status s = scan_check(&r);
    if (s != EMB_OK) return s;
    const size_t el = dtype == EMB_BF16 ? 2 : 4;
    if (rows == 0) return EMB_OK;
    if (!x || !gate || !state || !y) return fail(EMB_ERR_INVALID_ARG, "recurrence step: x, gate, state and y must be given");
    if (!aligned(x, el) || !aligned(gate, el) || !aligned(y, el) || !aligned(state, 4))
        return fail(EMB_ERR_INVALID_ARG, "recurrence step: buffers must be aligned to their elements");
    const bool pairs = pairs_ok(&r, {y}) && aligned(state, 8);
    const int64_t items = rows * (pairs ? channels / 2 : channels);
    const int64_t blocks = (items + 255) / 256;
    if (blocks > 0x7FFFFFFF) return fail(EMB_ERR_UNSUPPORTED, "recurrence step: more than 2^31 - 1 blocks");
    const dim3 grid((unsigned)blocks), block(256);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == EMB_BF16 && pairs)
        hipLaunchKernelGGL((scan_step<uint16_t, 2>), grid, block, 0, st, static_cast<const uint16_t *>(x),
                           static_cast<const uint16_t *>(gate), x_stride, gate_stride, state,
                           static_cast<uint16_t *>(y), rows, (int64_t)channels);
    else if (dtype == EMB_BF16)
        hipLaunchKernelGGL((scan_step<uint16_t, 1>), grid, block, 0, st, static_cast<const uint16_t *>(x),
                           static_cast<const uint16_t *>(gate), x_stride, gate_stride, state,
                           static_cast<uint16_t *>(y), rows, (int64_t)channels);
    else if (pairs)
        hipLaunchKernelGGL((scan_step<float, 2>), grid, block, 0, st, static_cast<const float *>(x),
                           static_cast<const float *>(gate), x_stride, gate_stride, state, static_cast<float *>(y),
                           rows, (int64_t)channels);
    else
        hipLaunchKernelGGL((scan_step<float, 1>), grid, block, 0, st, static_cast<const float *>(x),
                           static_cast<const float *>(gate), x_stride, gate_stride, state, static_cast<float *>(y),
                           rows, (int64_t)channels);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(EMB_ERR_HIP, std::string("recurrence step launch: ") + hipGetErrorString(e));
    return EMB_OK;
}
