// recurrence.hip -- the gated linear recurrence over jagged sequences,
//   a_t = sigmoid(gate_t),  h_t = a_t h_(t-1) + (1 - a_t) x_t  in every channel,
// its backward pass and its one-step form.
#include <string>

#include "sequence.h"

namespace emb {

constexpr int kSteps = 8;        // consecutive rows a half wavefront holds in registers; the
                                 // forward saves the state before every such group
constexpr int kWaves = 8;        // most wavefronts of a workgroup
constexpr int kChunk = 512;      // rows per chunk of a split scan (256 and 1024: no faster)

struct ScanArgs {
    const void *x, *gate;        // [n, channels], rows xs / gs elements apart
    int64_t xs, gs;
    const int32_t *off;          // [samples + 1]
    const uint8_t *mask;         // [n] or NULL
    const float *state;          // [samples, channels] or NULL
    void *y;                     // [n, channels]
    float *last;                 // [samples, channels]
    float *ckpt;                 // state before each group of kSteps rows, or NULL
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
    typedef uint32_t Bits;
    static __device__ __forceinline__ void open(Raw r, float *v) { v[0] = r; }
    static __device__ __forceinline__ Raw pack(const float *v) { return v[0]; }
};
template <>
struct Chan<float, 2> {
    typedef float2 Raw;          // in the one-step form, whose rows lie in plain memory
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
    typedef uint16_t Bits;
    static __device__ __forceinline__ void open(Raw r, float *v) { v[0] = bf16_lo(r); }
    static __device__ __forceinline__ Raw pack(const float *v) { return bf16_rne(v[0]); }
};
template <>
struct Chan<uint16_t, 2> {
    typedef uint32_t Raw;
    typedef uint32_t Bits;
    static __device__ __forceinline__ void open(Raw r, float *v)
    {
        v[0] = bf16_lo(r);
        v[1] = bf16_hi(r);
    }
    static __device__ __forceinline__ Raw pack(const float *v) { return bf16x2_rne(v[0], v[1]); }
};

__device__ __forceinline__ uint32_t buf_load(__amdgpu_buffer_rsrc_t r, int at, uint32_t)
{
    return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
}
__device__ __forceinline__ uint16_t buf_load(__amdgpu_buffer_rsrc_t r, int at, uint16_t)
{
    return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
}
__device__ __forceinline__ void buf_store(__amdgpu_buffer_rsrc_t r, int at, uint32_t v)
{
    __builtin_amdgcn_raw_buffer_store_b32(v, r, at, 0, 0);
}
__device__ __forceinline__ void buf_store(__amdgpu_buffer_rsrc_t r, int at, uint16_t v)
{
    __builtin_amdgcn_raw_buffer_store_b16(v, r, at, 0, 0);
}
// The rows of a block of the walk in one tensor, through a buffer descriptor that ends
// with the sample (or chunk): rows past the end read zeros and drop stores, and so do
// lanes past the last channel, whose offset lies past every end.
template <typename T, int VEC>
struct Rows {
    typedef Chan<T, VEC> CH;
    __amdgpu_buffer_rsrc_t rsrc;
    int at, stride;
    __device__ __forceinline__ Rows(const void *p, int64_t stride_, int row, int rows, int first, int c, bool live)
    {
        stride = (int)stride_ * (int)sizeof(T);
        rsrc = row_buffer(static_cast<const T *>(p) + row * stride_, 0, rows * stride);
        at = live ? first * stride + c * (int)sizeof(T) : INT32_MIN;
        // one addition per row, where it is used: taken out of the walk's loop, the offsets of
        // all rows of all tensors would be 40 registers
        asm volatile("" : "+v"(at));
    }
    // (an offset past the end stays one: rows and strides keep it below 2^31)
    __device__ __forceinline__ typename CH::Raw load(int i) const
    {
        return __builtin_bit_cast(typename CH::Raw, buf_load(rsrc, at + i * stride, typename CH::Bits{}));
    }
    __device__ __forceinline__ void store(int i, const float *v) const
    {
        buf_store(rsrc, at + i * stride, __builtin_bit_cast(typename CH::Bits, CH::pack(v)));
    }
};

// Which rows a workgroup walks: one sample, or one chunk of one.
struct ScanSpan {
    int begin, end;          // rows
    int first;               // first row of the sample
    int tile, tile0;         // chunk number, that of the sample's first chunk
    int chunks;              // of the sample
    int seg;
};

__device__ __forceinline__ bool scan_span(const ScanArgs &A, int block, ScanSpan &s)
{
    s.tile = block;
    if (A.chunk == 0) {
        s.seg = block;
        s.tile0 = block;
        s.chunks = 1;
        s.first = s.begin = uniform(seg_edge(A.off, A.samples, (int)A.n, s.seg));
        s.end = max(uniform(seg_edge(A.off, A.samples, (int)A.n, s.seg + 1)), s.begin);
        return true;
    }
    const SegTile t = seg_find<kChunk>(A.off, (int)A.n, nullptr, 0, A.samples, 1, block);
    s.seg = t.seg;
    s.first = t.base;
    s.tile0 = t.base / kChunk + t.seg;
    s.chunks = (t.rows + kChunk - 1) / kChunk;
    s.begin = t.base + t.row0;
    s.end = t.row0 + kChunk < t.rows ? s.begin + kChunk : t.base + t.rows;
    // an empty sample keeps its first chunk: it hands the state through
    return t.row0 < t.rows || (t.rows == 0 && t.row0 == 0);
}

// The saved state of the group of kSteps rows that begins at `row`
__device__ __forceinline__ int64_t saved_row(const ScanSpan &s, int row)
{
    return (int64_t)s.first / kSteps + s.seg + (row - s.first) / kSteps;
}

enum { kScanWhole = 0, kScanSum = 1, kScanApply = 2 };

// the other half's value of the same lane & 31
__device__ __forceinline__ float other_half(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(lane_id() < 32 ? r[1] : r[0]);
}

// What the pairs (A, H) of the sample's chunks before this one (after it, in the
// backward) make of the state v: each half wavefront folds its share of the pairs, and
// the results meet in LDS.
template <int VEC, int W, bool REVERSE>
__device__ __forceinline__ void chunk_state(const ScanArgs &A, const ScanSpan &s, int unit, int c, bool live,
                                            float (&pa)[2 * W][32 * VEC], float (&ph)[2 * W][32 * VEC], float *v)
{
    const int here = s.tile - s.tile0, n = max(REVERSE ? s.chunks - 1 - here : here, 0);
    const int i0 = n * unit / (2 * W), i1 = n * (unit + 1) / (2 * W), hl = lane_id() & 31;
    const int64_t C = A.channels;
    float a[VEC], h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; e++) {
        a[e] = 1.f;
        h[e] = 0.f;
    }
    constexpr int kAhead = 8;    // pairs loaded before the first is needed
    for (int i = i0; i < i1; i += kAhead) {
        float ra[kAhead][VEC], rh[kAhead][VEC];
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            const int k = i + j < i1 ? i + j : i1 - 1;
            const int64_t t = (s.tile0 + (REVERSE ? s.chunks - 1 - k : k)) * C + (live ? c : 0);
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                ra[j][e] = *gp(A.sum_a + t + e);
                rh[j][e] = *gp(A.sum_h + t + e);
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
        pa[unit][hl * VEC + e] = a[e];
        ph[unit][hl * VEC + e] = h[e];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2 * W; u++)
#pragma unroll
        for (int e = 0; e < VEC; e++) v[e] = fmaf(pa[u][hl * VEC + e], v[e], ph[u][hl * VEC + e]);
    __syncthreads();
}

// rows that nobody owns give zero
template <typename T, int VEC, int W>
__device__ __forceinline__ void zero_rows(void *p, const ScanSpan &s, int64_t C, int unit, int c, bool live)
{
    const float z[VEC] = {};
    for (int t = s.begin; t < s.end; t += 2 * W) {
        const Rows<T, VEC> r(p, C, t, min(s.end - t, 2 * W), unit, c, live);
        r.store(0, z);
    }
}

// W wavefronts walk a sample (or chunk) in blocks of 2 W kSteps rows: each half
// wavefront loads its own kSteps rows of 32 * VEC channels (so a load covers two rows,
// and 64 channels of bf16 are a workgroup's: there are enough workgroups to even out
// samples of very different lengths), scans them from a zero state into (A, H) with
// h_out = A h_in + H; two halves make a wavefront's pair, the W pairs meet in LDS, and
// each half applies its rows from the state that the pairs before it give.  One pass
// over the data; the state stays in fp32 registers.  Rows past the end and masked ones
// count as a = 1, x = 0; the next block's rows are loaded before this block's last step.
// 256 samples of 200..2000 rows, 256 channels, bf16, mask and states: 106 us, 4.0 TB/s of
// its 423 MB (a large copy: 5.5), in registers for four wavefronts a SIMD (six: spills,
// 212 us).  An exponential and a reciprocal an element keep the vector units half busy,
// and samples of unequal length leave the chip emptying at the end.  Cut (two passes) one
// fp32 sample of 65537 rows and 384 channels takes 42 us and 54 us.
template <typename T, int VEC, int W, int PHASE>
__global__ __launch_bounds__(64 * W, W == 1 ? 1 : 4) void scan_forward(ScanArgs A)
{
    typedef Chan<T, VEC> CH;
    typedef typename CH::Raw Raw;
    constexpr int kRows = 2 * W * kSteps;
    __shared__ float pa[2 * W][32 * VEC], ph[2 * W][32 * VEC];
    const int lane = lane_id(), hl = lane & 31, half = lane >> 5, w = uniform((int)(threadIdx.x >> 6));
    const int unit = 2 * w + half, c = (blockIdx.y * 32 + hl) * VEC;
    const bool live = c < A.channels;
    const int64_t C = A.channels;
    ScanSpan s;
    // the chunks' second pass begins with what the first read last (64 x 4096 rows: 437 -> 426 us)
    if (!scan_span(A, PHASE == kScanApply ? gridDim.x - 1 - blockIdx.x : blockIdx.x, s)) return;
    if (s.seg == 0 || s.seg == A.samples + 1) {
        if (PHASE != kScanSum) zero_rows<T, VEC, W>(A.y, s, C, unit, c, live);
        return;
    }
    float h[VEC], ta[VEC];
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        h[v] = PHASE != kScanSum && A.state && live ? A.state[(s.seg - 1) * C + c + v] : 0.f;
        ta[v] = 1.f;
    }
    if (PHASE == kScanApply) chunk_state<VEC, W, false>(A, s, unit, c, live, pa, ph, h);

    Raw xn[kSteps], gn[kSteps];
    int keep = 0;
    auto load = [&](int t0) {
        const int row = t0 + unit * kSteps + (hl & (kSteps - 1));
        keep = row < s.end ? (A.mask ? *gp(A.mask + row) : 1) : 0;
        const int rows = min(s.end - t0, kRows);
        const Rows<T, VEC> x(A.x, A.xs, t0, rows, unit * kSteps, c, live);
        const Rows<T, VEC> g(A.gate, A.gs, t0, rows, unit * kSteps, c, live);
#pragma unroll
        for (int i = 0; i < kSteps; i++) {
            xn[i] = x.load(i);
            gn[i] = g.load(i);
        }
    };
    if (s.begin < s.end) load(s.begin);
    int buf = 0;             // the pairs lie in either half in turn: one barrier a block
    for (int t0 = s.begin; t0 < s.end; t0 += kRows, buf ^= W) {
        const uint64_t all = __ballot(keep != 0);
        const uint32_t bits = half ? (uint32_t)(all >> 32) : (uint32_t)all;
        float xs[kSteps][VEC], as[kSteps][VEC], la[VEC], lh[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            la[v] = 1.f;
            lh[v] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kSteps; i++) {
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
        if (t0 + kRows < s.end) load(t0 + kRows);
        float oa[VEC], oh[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            oa[v] = other_half(la[v]);
            oh[v] = other_half(lh[v]);
            // half 0's pair, then half 1's
            if (half == 0) {
                pa[buf + w][hl * VEC + v] = la[v] * oa[v];
                ph[buf + w][hl * VEC + v] = fmaf(oa[v], lh[v], oh[v]);
            }
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
                const float ua = pa[buf + u][hl * VEC + v];
                h[v] = fmaf(ua, h[v], ph[buf + u][hl * VEC + v]);
                if (PHASE == kScanSum) ta[v] *= ua;
            }
        if (PHASE == kScanSum) continue;
        const int mine = t0 + unit * kSteps;
        const bool save = A.ckpt && live && mine < s.end;
        const int64_t group = save ? saved_row(s, mine) * C + c : 0;
        const Rows<T, VEC> y(A.y, C, t0, min(s.end - t0, kRows), unit * kSteps, c, live);
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            if (half) in[v] = fmaf(oa[v], in[v], oh[v]);
            if (save) *gp(A.ckpt + group + v) = in[v];
        }
#pragma unroll
        for (int i = 0; i < kSteps; i++) {
#pragma unroll
            for (int v = 0; v < VEC; v++) in[v] = fmaf(as[i][v], in[v], xs[i][v]);
            y.store(i, in);
        }
    }
    if (!live || unit != 0) return;
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        if (PHASE == kScanWhole || (PHASE == kScanApply && s.tile - s.tile0 >= s.chunks - 1))
            A.last[(s.seg - 1) * C + c + v] = h[v];
        if (PHASE == kScanSum) {
            A.sum_a[s.tile * C + c + v] = ta[v];
            A.sum_h[s.tile * C + c + v] = h[v];
        }
    }
}

// The backward pass walks the same blocks from the last to the first.  With
// u_t = a_t g_t the carried quantity, g_t = dy_t + u_(t+1) is the gradient of h_t,
// again a linear recurrence.  The states h_(t-1) that dgate needs are scanned again
// from the saved state before each group of kSteps rows: an eighth of the states in
// fp32 is a quarter of what all of them in bf16 would cost, and exact.
// 128 samples of 200..2000 rows, 512 channels, bf16: 150 to 163 us, 4.4 to 4.8 TB/s of the
// 688 MB of x, gate, dy, dx and dgate and 34 MB of saved states (the forward that saves them
// 106 to 111 us); bounded as the forward is.  Cut, as above: 35 us and 84 us.
template <typename T, int VEC, int W, int PHASE>
__global__ __launch_bounds__(64 * W, W == 1 ? 1 : 4) void scan_backward(ScanArgs A)
{
    typedef Chan<T, VEC> CH;
    typedef typename CH::Raw Raw;
    constexpr int kRows = 2 * W * kSteps;
    __shared__ float pa[2 * W][32 * VEC], ph[2 * W][32 * VEC];
    const int lane = lane_id(), hl = lane & 31, half = lane >> 5, w = uniform((int)(threadIdx.x >> 6));
    const int unit = 2 * w + half, c = (blockIdx.y * 32 + hl) * VEC;
    const bool live = c < A.channels;
    const int64_t C = A.channels;
    ScanSpan s;
    if (!scan_span(A, PHASE == kScanApply ? gridDim.x - 1 - blockIdx.x : blockIdx.x, s)) return;
    if (s.seg == 0 || s.seg == A.samples + 1) {
        if (PHASE != kScanSum) {
            zero_rows<T, VEC, W>(A.dx, s, C, unit, c, live);
            zero_rows<T, VEC, W>(A.dgate, s, C, unit, c, live);
        }
        return;
    }
    float u[VEC], ta[VEC];
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        u[v] = PHASE != kScanSum && A.dlast && live ? A.dlast[(s.seg - 1) * C + c + v] : 0.f;
        ta[v] = 1.f;
    }
    if (PHASE == kScanApply) chunk_state<VEC, W, true>(A, s, unit, c, live, pa, ph, u);

    const int blocks = (s.end - s.begin + kRows - 1) / kRows;
    Raw xn[kSteps], gn[kSteps], dn[kSteps];
    float hn[VEC];
    int keep = 0;
    auto load = [&](int b) {
        const int t0 = s.begin + b * kRows, mine = t0 + unit * kSteps, row = mine + (hl & (kSteps - 1));
        keep = row < s.end ? (A.mask ? *gp(A.mask + row) : 1) : 0;
        const int rows = min(s.end - t0, kRows);
        const Rows<T, VEC> x(A.x, A.xs, t0, rows, unit * kSteps, c, live);
        const Rows<T, VEC> g(A.gate, A.gs, t0, rows, unit * kSteps, c, live);
        const Rows<T, VEC> d(A.dy, C, t0, rows, unit * kSteps, c, live);
#pragma unroll
        for (int i = 0; i < kSteps; i++) {
            if (PHASE != kScanSum) xn[i] = x.load(i);
            gn[i] = g.load(i);
            dn[i] = d.load(i);
        }
        if (PHASE == kScanSum) return;
        const int64_t group = saved_row(s, mine < s.end ? mine : s.begin) * C + (live ? c : 0);
#pragma unroll
        for (int v = 0; v < VEC; v++) hn[v] = *gp(A.ckpt + group + v);
    };
    if (blocks) load(blocks - 1);
    int buf = 0;             // the pairs lie in either half in turn: one barrier a block
    for (int b = blocks - 1; b >= 0; b--, buf ^= W) {
        const int t0 = s.begin + b * kRows;
        const uint64_t all = __ballot(keep != 0);
        const uint32_t bits = half ? (uint32_t)(all >> 32) : (uint32_t)all;
        // x and dy stay as they lie in memory until they are needed: half the registers in bf16
        Raw xr[kSteps], dr[kSteps];
        float as[kSteps][VEC], na[kSteps][VEC], hin[VEC];
        float la[VEC], lu[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            la[v] = 1.f;
            lu[v] = 0.f;
            hin[v] = PHASE != kScanSum ? hn[v] : 0.f;
        }
#pragma unroll
        for (int i = kSteps - 1; i >= 0; i--) {
            const bool on = bits >> i & 1;
            float d[VEC];
            CH::open(gn[i], as[i]);
            CH::open(dn[i], d);          // zero past the end
            dr[i] = dn[i];
            if (PHASE != kScanSum) xr[i] = on ? xn[i] : Raw{};
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                sigmoid_pair(on ? as[i][v] : INFINITY, as[i][v], na[i][v]);
                lu[v] = as[i][v] * (d[v] + lu[v]);
                la[v] *= as[i][v];
            }
        }
        if (b > 0) load(b - 1);
        float oa[VEC], ou[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            oa[v] = other_half(la[v]);
            ou[v] = other_half(lu[v]);
            // half 1's pair, then half 0's
            if (half == 0) {
                pa[buf + w][hl * VEC + v] = la[v] * oa[v];
                ph[buf + w][hl * VEC + v] = fmaf(la[v], ou[v], lu[v]);
            }
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
                const float pv = pa[buf + p][hl * VEC + v];
                u[v] = fmaf(pv, u[v], ph[buf + p][hl * VEC + v]);
                if (PHASE == kScanSum) ta[v] *= pv;
            }
        if (PHASE == kScanSum) continue;
#pragma unroll
        for (int v = 0; v < VEC; v++)
            if (!half) in[v] = fmaf(oa[v], in[v], ou[v]);
        // forward again: h_(t-1) - x_t, what dgate multiplies
        float diff[kSteps][VEC];
#pragma unroll
        for (int i = 0; i < kSteps; i++) {
            float x[VEC];
            CH::open(xr[i], x);
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                const float before = hin[v];
                hin[v] = fmaf(as[i][v], before, na[i][v] * x[v]);
                diff[i][v] = before - x[v];
            }
        }
        const int rows = min(s.end - t0, kRows);
        const Rows<T, VEC> dx(A.dx, C, t0, rows, unit * kSteps, c, live);
        const Rows<T, VEC> dg(A.dgate, C, t0, rows, unit * kSteps, c, live);
#pragma unroll
        for (int i = kSteps - 1; i >= 0; i--) {
            float gx[VEC], gg[VEC], d[VEC];
            CH::open(dr[i], d);
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                const float g = d[v] + in[v];
                in[v] = as[i][v] * g;
                gx[v] = na[i][v] * g;                        // a masked row has na = 0
                gg[v] = as[i][v] * diff[i][v] * gx[v];
            }
            dx.store(i, gx);
            dg.store(i, gg);
        }
    }
    if (!live || unit != 0) return;
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        if (A.dstate && (PHASE == kScanWhole || (PHASE == kScanApply && s.tile == s.tile0)))
            A.dstate[(s.seg - 1) * C + c + v] = u[v];
        if (PHASE == kScanSum) {
            A.sum_a[s.tile * C + c + v] = ta[v];
            A.sum_h[s.tile * C + c + v] = u[v];
        }
    }
}

// One row for each of a batch of states.  2.3 us for 64 states of 256 channels: a launch.
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
    int waves;
    int32_t chunk;               // cut samples into chunks
    int64_t tiles, saved;
};

// How many wavefronts walk a sample, and whether samples are cut.  Times in us of a
// training step (forward and backward) in bf16 over 256 channels, measured.
// A workgroup's block of rows is 16 per wavefront, and a sample shorter than that
// wastes the rest (about 256000 rows in all):
//   mean length   4    16    32    64   128   256
//   1 wavefront  389   236   248   271   320   378
//   4           1383   439   285   236   257   288
//   8           3405   996   553   350   268   271
// Cutting reads x and gate (the backward: dy and gate) twice and costs two more launches,
// but lets few samples fill the chip (samples x mean length, whole / cut): 1 x 65536
// 2038 / 93, 16 x 8192 281 / 169; 64 x 4096 of very different lengths 707 / 432; and the
// other side 32 x 512 25 / 63, 100 x 1024 of equal lengths 86 / 140, of very different
// ones 210 / 155.  The lengths themselves are on the device: only their mean is known here.
ScanPlan scan_plan(const emb_recurrence *r)
{
    ScanPlan p{};
    const int64_t mean = r->samples ? r->n / r->samples : 0;
    const int per = r->dtype == EMB_BF16 ? 64 : 32;      // channels a workgroup
    const int64_t items = (int64_t)r->samples * ((r->channels + per - 1) / per);
    p.waves = mean <= 32 ? 1 : mean <= 128 ? 4 : kWaves;
    p.chunk = mean >= 1024 && items <= 256 && items * 8 <= mean;
    p.tiles = p.chunk ? seg_tiles(r->n, r->samples, 1, kChunk) : r->samples + 2;
    p.saved = seg_tiles(r->n, r->samples, 1, kSteps);
    return p;
}

// the rows of a block lie within the 2^31 bytes that a buffer descriptor reaches
constexpr int64_t kStrideMost = (int64_t(1) << 21) - 1;
static_assert(kStrideMost * 4 * 2 * kWaves * kSteps < int64_t(1) << 31, "a block of rows fits a descriptor");

// The stride of a single row leads nowhere, and may be anything (a transposed column's is 1,
// a broadcast row's 0).  The kernels take the length of the rows' buffers from it, so there
// it becomes the row's own length.
emb_recurrence with_strides(const emb_recurrence *r)
{
    emb_recurrence own = *r;
    if (own.n <= 1) own.x_stride = own.gate_stride = own.channels;
    return own;
}

emb_status scan_check(const emb_recurrence *r)
{
    if (r->dtype != EMB_F32 && r->dtype != EMB_BF16) return fail(EMB_ERR_INVALID_ARG, "recurrence: unknown dtype");
    if (r->samples < 0 || r->n < 0) return fail(EMB_ERR_INVALID_ARG, "recurrence: samples and n must be >= 0");
    if (r->channels <= 0) return fail(EMB_ERR_INVALID_ARG, "recurrence: channels must be >= 1");
    if (r->channels > (1 << 20)) return fail(EMB_ERR_UNSUPPORTED, "recurrence: channels must be <= 2^20");
    if (r->n > kRowsMost || r->samples > (1 << 30))
        return fail(EMB_ERR_UNSUPPORTED, "recurrence: n must be <= 2^31 - 65536 and samples <= 2^30");
    if (r->x_stride < r->channels || r->gate_stride < r->channels)
        return fail(EMB_ERR_INVALID_ARG, "recurrence: row strides must be >= channels");
    if (r->x_stride > kStrideMost || r->gate_stride > kStrideMost)
        return fail(EMB_ERR_UNSUPPORTED, "recurrence: row strides must be < 2^21");
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

// a launch's threads in one dimension are counted in 32 bits
constexpr int64_t kThreadsMost = (int64_t(1) << 32) - 1;

template <typename T, int VEC, int W, int PHASE>
void scan_launch_p(const ScanArgs &A, bool backward, hipStream_t st)
{
    const int64_t blocks = (A.channels + 32 * VEC - 1) / (32 * VEC);
    const dim3 grid((unsigned)A.tiles, (unsigned)blocks), block(64 * W);
    if (backward) hipLaunchKernelGGL((scan_backward<T, VEC, W, PHASE>), grid, block, 0, st, A);
    else hipLaunchKernelGGL((scan_forward<T, VEC, W, PHASE>), grid, block, 0, st, A);
}

template <typename T, int VEC>
emb_status scan_launch_v(const ScanArgs &A, int waves, bool backward, hipStream_t st)
{
    if (A.tiles > kThreadsMost / (64 * waves))
        return fail(EMB_ERR_UNSUPPORTED, "recurrence: too many samples for one launch");
    if (A.chunk) {                       // samples long enough for kWaves
        scan_launch_p<T, VEC, kWaves, kScanSum>(A, backward, st);
        scan_launch_p<T, VEC, kWaves, kScanApply>(A, backward, st);
    } else if (waves == 1) scan_launch_p<T, VEC, 1, kScanWhole>(A, backward, st);
    else if (waves == 4) scan_launch_p<T, VEC, 4, kScanWhole>(A, backward, st);
    else scan_launch_p<T, VEC, kWaves, kScanWhole>(A, backward, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(EMB_ERR_HIP, std::string("recurrence launch: ") + hipGetErrorString(e));
    return EMB_OK;
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

extern "C" emb_status emb_recurrence_query(const emb_recurrence *desc, int64_t *saved_rows, size_t *workspace_bytes)
{
    if (!desc) return fail(EMB_ERR_INVALID_ARG, "recurrence descriptor is NULL");
    const emb_recurrence own = with_strides(desc), *r = &own;
    const emb_status s = scan_check(r);
    if (s != EMB_OK) return s;
    if (!saved_rows || !workspace_bytes) return fail(EMB_ERR_INVALID_ARG, "recurrence: output pointers must be given");
    const ScanPlan p = scan_plan(r);
    *saved_rows = p.saved;
    *workspace_bytes = scan_workspace(r, p);
    return EMB_OK;
}

extern "C" emb_status emb_recurrence_forward(const emb_recurrence *desc, void *y, float *last, float *saved,
                                             void *workspace, size_t workspace_bytes, void *stream)
{
    if (!desc) return fail(EMB_ERR_INVALID_ARG, "recurrence descriptor is NULL");
    const emb_recurrence own = with_strides(desc), *r = &own;
    emb_status s = scan_check(r);
    if (s == EMB_OK) s = scan_pointers(r);
    if (s != EMB_OK) return s;
    const size_t el = r->dtype == EMB_BF16 ? 2 : 4;
    if ((r->n && !y) || (r->samples && !last) || !aligned(y, el) || !aligned(last, 4) || !aligned(saved, 4))
        return fail(EMB_ERR_INVALID_ARG, "recurrence: y and last must be given and aligned");
    const ScanPlan p = scan_plan(r);
    if (workspace_bytes < scan_workspace(r, p) || (scan_workspace(r, p) && !aligned(workspace, 256)))
        return fail(EMB_ERR_WORKSPACE, "recurrence: the workspace is smaller than the query returned, or not 256-byte aligned");
    if (scan_workspace(r, p) && !workspace) return fail(EMB_ERR_WORKSPACE, "recurrence: workspace is NULL");
    ScanArgs A = scan_args(r, p, workspace);
    A.y = y;
    A.last = last;
    A.ckpt = saved;
    return scan_launch(r, A, p.waves, pairs_ok(r, {y}), false, stream);
}

extern "C" emb_status emb_recurrence_backward(const emb_recurrence *desc, const float *saved, const void *dy,
                                              const float *dlast, void *dx, void *dgate, float *dstate,
                                              void *workspace, size_t workspace_bytes, void *stream)
{
    if (!desc) return fail(EMB_ERR_INVALID_ARG, "recurrence descriptor is NULL");
    const emb_recurrence own = with_strides(desc), *r = &own;
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
    if (scan_workspace(r, p) && !workspace) return fail(EMB_ERR_WORKSPACE, "recurrence: workspace is NULL");
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
    r = with_strides(&r);
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
    if (blocks > kThreadsMost / 256)
        return fail(EMB_ERR_UNSUPPORTED, "recurrence step: more than 2^32 - 256 channels or pairs of them");
    const dim3 grid((unsigned)blocks), block(256);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == EMB_BF16 && pairs)
        hipLaunchKernelGGL((scan_step<uint16_t, 2>), grid, block, 0, st, static_cast<const uint16_t *>(x),
                           static_cast<const uint16_t *>(gate), r.x_stride, r.gate_stride, state,
                           static_cast<uint16_t *>(y), rows, (int64_t)channels);
    else if (dtype == EMB_BF16)
        hipLaunchKernelGGL((scan_step<uint16_t, 1>), grid, block, 0, st, static_cast<const uint16_t *>(x),
                           static_cast<const uint16_t *>(gate), r.x_stride, r.gate_stride, state,
                           static_cast<uint16_t *>(y), rows, (int64_t)channels);
    else if (pairs)
        hipLaunchKernelGGL((scan_step<float, 2>), grid, block, 0, st, static_cast<const float *>(x),
                           static_cast<const float *>(gate), r.x_stride, r.gate_stride, state, static_cast<float *>(y),
                           rows, (int64_t)channels);
    else
        hipLaunchKernelGGL((scan_step<float, 1>), grid, block, 0, st, static_cast<const float *>(x),
                           static_cast<const float *>(gate), r.x_stride, r.gate_stride, state, static_cast<float *>(y),
                           rows, (int64_t)channels);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(EMB_ERR_HIP, std::string("recurrence step launch: ") + hipGetErrorString(e));
    return EMB_OK;
}
