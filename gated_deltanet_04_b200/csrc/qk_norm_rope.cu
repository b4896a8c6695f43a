// RMS norm of every query and key head row and the rotation of its first `rot`
// dimensions by the token's positions, in one pass over memory, with its
// backward pass: what feeds a linear attention (or attention) layer, as the
// short convolution with its norm feeds the gated delta rule.
//
// Row x of one (token, head), D elements:
//     r = (mean(x^2) + eps)^(-1/2),  y = x r w,  z = Rot(y)
// Rot turns the pair of frequency i, (y[i], y[i + rot/2]) or, interleaved,
// (y[2i], y[2i + 1]), by the angle pos[axis(i)] inv_freq[i].  Backward, with
// dy = Rot^T(dz), n = x r:
//     dw = sum over rows of dy n,   dx = r (dy w - n mean(dy w n))
//
// Angles: a far position times a frequency needs more than 24 bits, so the
// number of whole turns is taken off in fp64; sine and cosine are then fp32
// on at most half a turn.  A CTA computes them once per token it covers and
// keeps them in shared memory for all its heads.
//
// Bound by HBM bandwidth, x read once and z written once (backward: x and dz
// read, dx written), and nearly by instruction issue: a row is spread over D / 8
// lanes with two pieces of 4 elements each, chosen so that a lane holds both of
// every pair it turns, and the arithmetic is on pairs of floats.  (With 8
// consecutive elements per lane and partners exchanged by shuffles it took twice
// the instructions and twice the time.)  A CTA takes kIter rows per lane group
// with all their loads in flight before the angles are computed.
#include "gdn_internal.cuh"
#include "sm100.cuh"
#include "trace.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxAxes = 4;
constexpr int kBackwardCtas = 444;  // persistent grid of the backward pass (3 per SM of 148)

// The queries or the keys: a CTA works on one side only, so that its heads,
// weights and pointers are uniform.
struct Side {
    const void *x, *dz;        // inputs; backward: gradients of the outputs
    void *out;                 // outputs, or the gradients of x
    const float *w;            // [D] or null (ones)
    uint32_t x_step, out_step, dz_step;  // bytes per token
    int32_t H;
    uint32_t inv_h;            // ceil(2^32 / H) (H > 1)
    int64_t rows;              // T * H
    uint32_t ctas;
};

struct RopeArgs {
    Side side[2];
    float *dw_part;            // backward: [CTAs][D] or null
    const int32_t *pos;        // [axes][T]
    const float *inv_freq;     // [rot / 2]
    int32_t last[kMaxAxes];    // frequency i belongs to the first axis with i < last[axis]
    float eps;
    int32_t rot, interleaved;
    uint32_t inv_half;         // ceil(2^32 / (rot / 2))
    int32_t blocks;            // blocks of kIter rows per lane group that share their angles
    int64_t T;
};

using sm100::ffma2;
using sm100::fmul2;

__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }

// Where a lane's 8 elements of a row are: 4 from p0, 4 from p1.  Rotated
// halves: the same 4 of the lower and of the upper half; otherwise (interleaved
// pairs, elements that are not rotated) 8 in a row.  `angle`: the lane's first
// frequency, or -1.
struct Pieces {
    int p0, p1, angle;
    __device__ __forceinline__ Pieces(int l, int rot, int interleaved) {
        const bool in = 8 * l < rot;
        p0 = in && !interleaved ? 4 * l : 8 * l;
        p1 = in && !interleaved ? rot / 2 + 4 * l : 8 * l + 4;
        angle = in ? 4 * l : -1;
    }
};

// A lane's two pieces of a row, as loaded, and as four pairs of floats.
template <class E>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
    uint2 a, b;
    __device__ __forceinline__ void load(const uint8_t *p, const Pieces &c) {
        a = *reinterpret_cast<const uint2 *>(p + 2 * c.p0);
        b = *reinterpret_cast<const uint2 *>(p + 2 * c.p1);
    }
    static __device__ __forceinline__ float2 wide(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
        f[0] = wide(a.x);
        f[1] = wide(a.y);
        f[2] = wide(b.x);
        f[3] = wide(b.y);
    }
    static __device__ __forceinline__ uint32_t narrow(float2 x) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(x.x, x.y);
        return *reinterpret_cast<const uint32_t *>(&t);
    }
    static __device__ __forceinline__ void store(uint8_t *p, const Pieces &c, const float2 (&f)[4]) {
        *reinterpret_cast<uint2 *>(p + 2 * c.p0) = make_uint2(narrow(f[0]), narrow(f[1]));
        *reinterpret_cast<uint2 *>(p + 2 * c.p1) = make_uint2(narrow(f[2]), narrow(f[3]));
    }
};
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const uint8_t *p, const Pieces &c) {
        a = *reinterpret_cast<const float4 *>(p + 4 * c.p0);
        b = *reinterpret_cast<const float4 *>(p + 4 * c.p1);
    }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
        f[0] = make_float2(a.x, a.y);
        f[1] = make_float2(a.z, a.w);
        f[2] = make_float2(b.x, b.y);
        f[3] = make_float2(b.z, b.w);
    }
    static __device__ __forceinline__ void store(uint8_t *p, const Pieces &c, const float2 (&f)[4]) {
        *reinterpret_cast<float4 *>(p + 4 * c.p0) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        *reinterpret_cast<float4 *>(p + 4 * c.p1) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
};

template <int N>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int off = N / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// cos and sin of tokens t0 .. t0 + n - 1 into [token][rot/2] each.
__device__ __forceinline__ void angles(const RopeArgs &a, int64_t t0, uint32_t n, float *cosines, float *sines) {
    const uint32_t half = (uint32_t)a.rot / 2;
    for (uint32_t i = threadIdx.x; i < n * half; i += kThreads) {
        const uint32_t tok = __umulhi(i, a.inv_half), f = i - tok * half;  // i half < 2^32: exact
        int axis = 0;
        while (axis < kMaxAxes - 1 && (int)f >= a.last[axis]) ++axis;
        // whole turns removed in fp64: |turns| < 2^31 leaves 2^-22 of a turn at worst
        const double turns = (double)a.pos[axis * a.T + t0 + tok] * ((double)a.inv_freq[f] * 0.15915494309189533577);
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        cosines[i] = c;
        sines[i] = s;
    }
}

// The lane's pieces of an fp32 row (weights).
__device__ __forceinline__ void load_pieces(const float *p, const Pieces &c, float2 (&f)[4]) {
    const float4 a = *reinterpret_cast<const float4 *>(p + c.p0), b = *reinterpret_cast<const float4 *>(p + c.p1);
    f[0] = make_float2(a.x, a.y);
    f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y);
    f[3] = make_float2(b.z, b.w);
}

// Turns the lane's pairs by its token's angles; sign = -1 turns them back.
__device__ __forceinline__ void rotate(float2 (&y)[4], const Pieces &c, const float *cosines, const float *sines,
                                       int interleaved, float sign) {
    if (c.angle < 0) return;
    const float4 c4 = *reinterpret_cast<const float4 *>(cosines + c.angle);
    const float4 s4 = *reinterpret_cast<const float4 *>(sines + c.angle);
    if (interleaved) {
        const float cv[4] = {c4.x, c4.y, c4.z, c4.w}, sv[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float ss = sign * sv[j];
            y[j] = make_float2(y[j].x * cv[j] - y[j].y * ss, y[j].y * cv[j] + y[j].x * ss);
        }
        return;
    }
    const float2 cc[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
    const float2 ss[2] = {fmul2(make_float2(s4.x, s4.y), splat(sign)), fmul2(make_float2(s4.z, s4.w), splat(sign))};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float2 lo = y[j], hi = y[2 + j];
        y[j] = ffma2(lo, cc[j], fmul2(hi, make_float2(-ss[j].x, -ss[j].y)));
        y[2 + j] = ffma2(hi, cc[j], fmul2(lo, ss[j]));
    }
}

__device__ __forceinline__ float dot8(const float2 (&a)[4], const float2 (&b)[4]) {
    float2 s = fmul2(a[0], b[0]);
#pragma unroll
    for (int j = 1; j < 4; ++j) s = ffma2(a[j], b[j], s);
    return s.x + s.y;
}

// A CTA's rows of its side: `first` and the following ones, as tokens and heads.
struct Rows {
    int64_t t0;     // token of the first row
    uint32_t h0;    // its head
    uint32_t n;     // rows
    uint32_t n_tok;
    __device__ __forceinline__ Rows(const Side &d, int64_t first, int per) {
        // (a 64-bit division only where 32 bits do not hold the row)
        t0 = d.rows >> 32 ? first / d.H : (int64_t)((uint32_t)first / (uint32_t)d.H);
        h0 = (uint32_t)(first - t0 * d.H);
        n = (uint32_t)(d.rows - first < per ? d.rows - first : per);
        n_tok = (h0 + n - 1) / (uint32_t)d.H + 1;
    }
};
// Row r of them: its token (from t0) and its head.
struct Row {
    uint32_t tok, h;
    __device__ __forceinline__ Row(const Side &d, const Rows &rows, uint32_t r) {
        const uint32_t x = rows.h0 + r;  // x H < 2^32: the product with ceil(2^32 / H) divides exactly
        tok = d.H == 1 ? x : __umulhi(x, d.inv_h);
        h = x - tok * (uint32_t)d.H;
    }
    // from a pointer to token t0
    template <class E, int D, class P>
    __device__ __forceinline__ P *at(P *base, uint32_t step) const {
        return base + (uint64_t)tok * step + h * (uint32_t)(D * sizeof(E));
    }
};

// A CTA's rows go in a.blocks blocks of kIter rows per lane group: the next
// block's loads are in flight while one is computed, and the angles of all their
// tokens are computed once, before the first.
template <class E, int D, int kIter>
__global__ void __launch_bounds__(kThreads) gdn_qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
    extern __shared__ __align__(16) float smem[];
    constexpr int LPR = D / 8, GROUPS = kThreads / LPR, kBlock = GROUPS * kIter;
    const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const bool key = blockIdx.x >= a.side[0].ctas;
    const Side &d = a.side[key];
    const Pieces c(l, a.rot, a.interleaved);
    const Rows rows(d, (int64_t)(blockIdx.x - (key ? a.side[0].ctas : 0u)) * (kBlock * a.blocks), kBlock * a.blocks);
    const uint8_t *in = static_cast<const uint8_t *>(d.x) + rows.t0 * d.x_step;
    uint8_t *out = static_cast<uint8_t *>(d.out) + rows.t0 * d.out_step;
    Vec8<E> next[kIter];
    auto load = [&](uint32_t r0) {
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const uint32_t r = r0 + i * GROUPS;
            if (r < rows.n) next[i].load(Row(d, rows, r).at<E, D>(in, d.x_step), c);
        }
    };
    load(grp);
    float2 wv[4] = {splat(1.f), splat(1.f), splat(1.f), splat(1.f)};
    if (d.w) load_pieces(d.w, c, wv);
    const int half = a.rot / 2;
    float *cosines = smem, *sines = smem + rows.n_tok * half;
    angles(a, rows.t0, rows.n_tok, cosines, sines);
    __syncthreads();
    for (uint32_t b0 = 0; b0 < rows.n; b0 += kBlock) {
        Vec8<E> x[kIter];
#pragma unroll
        for (int i = 0; i < kIter; ++i) x[i] = next[i];
        load(b0 + kBlock + grp);
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const uint32_t r = b0 + i * GROUPS + grp;
            const bool live = r < rows.n;  // every lane runs the shuffles
            const Row w(d, rows, live ? r : 0);
            float2 y[4];
            x[i].get(y);
            const float2 rms = splat(rsqrtf(group_sum<LPR>(dot8(y, y)) * (1.f / D) + a.eps));
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = fmul2(y[j], fmul2(rms, wv[j]));
            const int off = (int)w.tok * half;
            rotate(y, c, cosines + off, sines + off, a.interleaved, 1.f);
            if (live) Vec8<E>::store(w.at<E, D>(out, d.out_step), c, y);
        }
    }
}

// Persistent: a side's CTA b takes the rows of blocks b, b + ctas, ... (each
// a.blocks blocks, as above); each lane keeps its 8 columns of the weight's
// gradient in registers, summed over the CTA at the end and over the CTAs by a
// second kernel (a fixed order, no atomics).
template <class E, int D, int kIter>
__global__ void __launch_bounds__(kThreads, sizeof(E) == 2 ? 3 : 2)
    gdn_qk_norm_rope_backward_kernel(const __grid_constant__ RopeArgs a) {
    extern __shared__ __align__(16) float smem[];
    constexpr int LPR = D / 8, GROUPS = kThreads / LPR, kBlock = GROUPS * kIter;
    const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const bool key = blockIdx.x >= a.side[0].ctas;
    const Side &d = a.side[key];
    const Pieces c(l, a.rot, a.interleaved);
    const int half = a.rot / 2;
    float2 acc[4] = {splat(0.f), splat(0.f), splat(0.f), splat(0.f)};
    float2 wv[4] = {splat(1.f), splat(1.f), splat(1.f), splat(1.f)};
    if (d.w) load_pieces(d.w, c, wv);
    const int64_t per = (int64_t)kBlock * a.blocks;
    for (int64_t first = (blockIdx.x - (key ? a.side[0].ctas : 0u)) * per; first < d.rows; first += d.ctas * per) {
        const Rows rows(d, first, (int)per);
        const uint8_t *in = static_cast<const uint8_t *>(d.x) + rows.t0 * d.x_step;
        const uint8_t *grad = static_cast<const uint8_t *>(d.dz) + rows.t0 * d.dz_step;
        uint8_t *out = static_cast<uint8_t *>(d.out) + rows.t0 * d.out_step;
        Vec8<E> next_x[kIter], next_g[kIter];
        auto load = [&](uint32_t r0) {
#pragma unroll
            for (int i = 0; i < kIter; ++i) {
                const uint32_t r = r0 + i * GROUPS;
                if (r < rows.n) {
                    const Row w(d, rows, r);
                    next_x[i].load(w.at<E, D>(in, d.x_step), c);
                    next_g[i].load(w.at<E, D>(grad, d.dz_step), c);
                }
            }
        };
        load(grp);
        __syncthreads();  // the previous rows' angles have been read
        float *cosines = smem, *sines = smem + rows.n_tok * half;
        angles(a, rows.t0, rows.n_tok, cosines, sines);
        __syncthreads();
        for (uint32_t b0 = 0; b0 < rows.n; b0 += kBlock) {
            Vec8<E> x[kIter], g[kIter];
#pragma unroll
            for (int i = 0; i < kIter; ++i) {
                x[i] = next_x[i];
                g[i] = next_g[i];
            }
            load(b0 + kBlock + grp);
#pragma unroll
            for (int i = 0; i < kIter; ++i) {
                const uint32_t r = b0 + i * GROUPS + grp;
                const bool live = r < rows.n;  // every lane runs the shuffles
                const Row w(d, rows, live ? r : 0);
                float2 n[4], dy[4];
                x[i].get(n);
                g[i].get(dy);
                const float rms = rsqrtf(group_sum<LPR>(dot8(n, n)) * (1.f / D) + a.eps);
                const int off = (int)w.tok * half;
                rotate(dy, c, cosines + off, sines + off, a.interleaved, -1.f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    n[j] = fmul2(n[j], splat(rms));
                    if (live) acc[j] = ffma2(dy[j], n[j], acc[j]);
                    dy[j] = fmul2(dy[j], wv[j]);
                }
                const float2 dot = splat(-group_sum<LPR>(dot8(dy, n)) * (1.f / D));
#pragma unroll
                for (int j = 0; j < 4; ++j) dy[j] = fmul2(ffma2(n[j], dot, dy[j]), splat(rms));
                if (live) Vec8<E>::store(w.at<E, D>(out, d.out_step), c, dy);
            }
        }
    }
    if (!a.dw_part) return;
    // sum over the CTA's lane groups: [D] from GROUPS partials, in order
    __syncthreads();
    float *mine = smem + grp * D;
    *reinterpret_cast<float4 *>(mine + c.p0) = make_float4(acc[0].x, acc[0].y, acc[1].x, acc[1].y);
    *reinterpret_cast<float4 *>(mine + c.p1) = make_float4(acc[2].x, acc[2].y, acc[3].x, acc[3].y);
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kThreads) {
        float s = 0.f;
        for (int q = 0; q < GROUPS; ++q) s += smem[q * D + i];
        a.dw_part[(int64_t)blockIdx.x * D + i] = s;
    }
}

// A side's dw[d] = the sum over its CTAs of part[cta][d]: 32 columns a CTA, 8 warps
// over the rows, then the warps' sums in order.
__global__ void gdn_qk_norm_dw_kernel(const float *part, uint32_t ctas_q, uint32_t ctas_k, int D, float *dwq,
                                      float *dwk) {
    __shared__ float sums[8][32];
    const bool key = blockIdx.y;
    float *dst = key ? dwk : dwq;
    if (!dst) return;
    const uint32_t first = key ? ctas_q : 0, n = key ? ctas_k : ctas_q;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (d < D) {
#pragma unroll 8
        for (uint32_t c = warp; c < n; c += 8) s += part[(int64_t)(first + c) * D + d];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && d < D) {
        for (int w = 1; w < 8; ++w) s += sums[w][lane];
        dst[d] = s;
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool supported(int32_t D) { return D == 16 || D == 32 || D == 64 || D == 128 || D == 256; }

// Tokens a block of `rows` consecutive rows can touch.
int64_t tokens_of(int64_t rows, int32_t H) { return rows / H + 2; }

// Blocks of `block` rows per CTA, so that their angles are computed once: as many
// (up to 8) as keep `ctas` CTAs busy and the angles within 40 KB.
int blocks_per_cta(const RopeArgs &a, int64_t block, int64_t ctas) {
    const int64_t rows = a.side[0].rows + a.side[1].rows;
    const int32_t fewest = a.side[1].H > 0 && a.side[1].H < a.side[0].H ? a.side[1].H : a.side[0].H;
    int n = 1;
    while (n < 8 && rows >= block * 2 * n * ctas &&
           tokens_of(block * 2 * n, fewest) * a.rot * (int64_t)sizeof(float) <= 40 * 1024)
        n *= 2;
    return n;
}

// Shared memory for the angles of `per` rows of either side.
size_t angle_bytes(const RopeArgs &a, int64_t per) {
    const int32_t fewest = a.side[1].H > 0 && a.side[1].H < a.side[0].H ? a.side[1].H : a.side[0].H;
    return (size_t)tokens_of(per, fewest) * a.rot * sizeof(float);
}

template <class E, int D>
cudaError_t launch_forward(RopeArgs a, cudaStream_t s) {
    constexpr int GROUPS = kThreads / (D / 8);
    // two rows per lane group at a time once that still fills the GPU, one below (latency)
    const bool many = a.side[0].rows + a.side[1].rows >= (int64_t)GROUPS * 2 * 592;
    const int block = GROUPS * (many ? 2 : 1);
    a.blocks = many ? blocks_per_cta(a, block, 592) : 1;
    const int64_t per = (int64_t)block * a.blocks;
    for (Side &d : a.side) d.ctas = (uint32_t)((d.rows + per - 1) / per);
    auto *fn = many ? gdn_qk_norm_rope_kernel<E, D, 2> : gdn_qk_norm_rope_kernel<E, D, 1>;
    fn<<<a.side[0].ctas + a.side[1].ctas, kThreads, angle_bytes(a, per), s>>>(a);
    return cudaGetLastError();
}

template <class E, int D>
cudaError_t launch_backward(RopeArgs a, float *dwq, float *dwk, cudaStream_t s) {
    constexpr int GROUPS = kThreads / (D / 8), kIter = 2;
    const int block = GROUPS * kIter;
    a.blocks = blocks_per_cta(a, block, kBackwardCtas);
    const int64_t per = (int64_t)block * a.blocks;
    // CTAs for each side in proportion to its rows (one at least), no more than it has blocks
    const int64_t all = a.side[0].rows + a.side[1].rows;
    for (Side &d : a.side) {
        const int64_t blocks = (d.rows + per - 1) / per, share = (kBackwardCtas - 1) * d.rows / all;
        d.ctas = (uint32_t)(blocks < share ? blocks : share > 0 ? share : d.rows > 0);
    }
    size_t smem = angle_bytes(a, per);
    if (smem < (size_t)GROUPS * D * sizeof(float)) smem = (size_t)GROUPS * D * sizeof(float);
    gdn_qk_norm_rope_backward_kernel<E, D, kIter><<<a.side[0].ctas + a.side[1].ctas, kThreads, smem, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.dw_part) return e;
    gdn_qk_norm_dw_kernel<<<dim3((D + 31) / 32, 2), 256, 0, s>>>(a.dw_part, a.side[0].ctas, a.side[1].ctas, D, dwq,
                                                                dwk);
    return cudaGetLastError();
}

template <class E>
cudaError_t dispatch(const RopeArgs &a, int32_t D, bool backward, float *dwq, float *dwk, cudaStream_t s) {
    switch (D) {
        case 16: return backward ? launch_backward<E, 16>(a, dwq, dwk, s) : launch_forward<E, 16>(a, s);
        case 32: return backward ? launch_backward<E, 32>(a, dwq, dwk, s) : launch_forward<E, 32>(a, s);
        case 64: return backward ? launch_backward<E, 64>(a, dwq, dwk, s) : launch_forward<E, 64>(a, s);
        case 128: return backward ? launch_backward<E, 128>(a, dwq, dwk, s) : launch_forward<E, 128>(a, s);
        case 256: return backward ? launch_backward<E, 256>(a, dwq, dwk, s) : launch_forward<E, 256>(a, s);
    }
    return cudaErrorInvalidValue;
}

// Checks of what both directions share; fills the common part of `a`.
gdn_status common(RopeArgs &a, const void *xq, const void *xk, gdn_dtype dt, int64_t xq_stride,
                  int64_t xk_stride, const float *wq, const float *wk, float eps, const int32_t *positions,
                  int32_t axes, const int32_t *sections, const float *inv_freq, int32_t rot,
                  int32_t interleaved, int64_t T, int32_t Hq, int32_t Hk, int32_t D) {
    if (dt != GDN_DTYPE_BF16 && dt != GDN_DTYPE_F32) return GDN_ERR_INVALID_ARGUMENT;
    if (T < 0 || Hq <= 0 || Hk < 0 || D <= 0 || rot < 0 || rot > D || !(eps > 0.f))
        return GDN_ERR_INVALID_ARGUMENT;
    if (interleaved != 0 && interleaved != 1) return GDN_ERR_INVALID_ARGUMENT;
    if (T > 0 && (!xq || (Hk > 0 && !xk))) return GDN_ERR_INVALID_ARGUMENT;
    if (rot > 0) {
        if (axes < 1 || (T > 0 && (!positions || !inv_freq)) || (axes > 1 && !sections))
            return GDN_ERR_INVALID_ARGUMENT;
        if (axes > kMaxAxes) return GDN_ERR_UNSUPPORTED;
        int64_t sum = 0;
        for (int i = 0; i < kMaxAxes; ++i) {
            if (i < axes && sections) {
                if (sections[i] < 0) return GDN_ERR_INVALID_ARGUMENT;
                sum += sections[i];
            } else if (i < axes) {
                sum = rot / 2;
            }
            a.last[i] = (int32_t)(sum < rot / 2 ? sum : rot / 2);
        }
        if (sum != rot / 2) return GDN_ERR_INVALID_ARGUMENT;
    }
    const int64_t esz = dt == GDN_DTYPE_BF16 ? 2 : 4;
    if (xq_stride < (int64_t)Hq * D || (Hk > 0 && xk_stride < (int64_t)Hk * D)) return GDN_ERR_INVALID_ARGUMENT;
    // a token's bytes are 32-bit in the kernels
    if (xq_stride > 0x3fffffff || (Hk > 0 && xk_stride > 0x3fffffff)) return GDN_ERR_UNSUPPORTED;
    if ((xq_stride * esz) % 16 || (Hk > 0 && (xk_stride * esz) % 16)) return GDN_ERR_INVALID_ARGUMENT;
    if (!supported(D) || rot % 16 != 0 || Hq > 32768 - Hk) return GDN_ERR_UNSUPPORTED;
    // the grid's x dimension (divided: the product can pass 64 bits)
    if (T > ((int64_t)1 << 33) / (Hq + Hk)) return GDN_ERR_UNSUPPORTED;
    auto inverse = [](uint32_t n) { return (uint32_t)((((uint64_t)1 << 32) + n - 1) / n); };
    const int32_t heads[2] = {Hq, Hk};
    for (int z = 0; z < 2; ++z) {
        Side &d = a.side[z];
        d.x = z ? xk : xq;
        d.w = z ? wk : wq;
        d.x_step = heads[z] ? (uint32_t)((z ? xk_stride : xq_stride) * esz) : 0;
        d.H = heads[z];
        d.inv_h = heads[z] > 1 ? inverse((uint32_t)heads[z]) : 0;
        d.rows = T * (int64_t)heads[z];
        d.dz_step = d.out_step = (uint32_t)(heads[z] * (int64_t)D * esz);
    }
    a.inv_half = rot > 0 ? inverse((uint32_t)rot / 2) : 0;
    a.pos = positions; a.inv_freq = inv_freq; a.eps = eps;
    a.rot = rot; a.interleaved = interleaved;
    a.T = T;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

extern "C" {

gdn_status gdn_qk_norm_rope(const void *xq, const void *xk, gdn_dtype io_dtype, int64_t xq_stride,
                            int64_t xk_stride, const float *wq, const float *wk, float eps,
                            const int32_t *positions, int32_t axes, const int32_t *sections,
                            const float *inv_freq, int32_t rot, int32_t interleaved, int64_t T,
                            int32_t Hq, int32_t Hk, int32_t D, void *q, void *k, void *stream) {
    GDN_TRACE("gdn_qk_norm_rope");
    gdn::RopeArgs a{};
    if (gdn_status e = gdn::common(a, xq, xk, io_dtype, xq_stride, xk_stride, wq, wk, eps, positions, axes,
                                   sections, inv_freq, rot, interleaved, T, Hq, Hk, D))
        return e;
    if (T > 0 && (!q || (Hk > 0 && !k))) return GDN_ERR_INVALID_ARGUMENT;
    const void *all[] = {xq, xk, wq, wk, positions, inv_freq, q, k};
    for (const void *p : all)
        if (p && !gdn::aligned16(p)) return GDN_ERR_INVALID_ARGUMENT;
    const void *ins[] = {xq, xk, wq, wk, positions, inv_freq};
    for (const void *i : ins)
        if ((q && q == i) || (k && k == i)) return GDN_ERR_INVALID_ARGUMENT;
    if (q && q == k) return GDN_ERR_INVALID_ARGUMENT;
    if (T == 0) return GDN_OK;
    a.side[0].out = q;
    a.side[1].out = k;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = io_dtype == GDN_DTYPE_BF16
                              ? gdn::dispatch<__nv_bfloat16>(a, D, false, nullptr, nullptr, s)
                              : gdn::dispatch<float>(a, D, false, nullptr, nullptr, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_qk_norm_rope_backward_workspace_bytes(int32_t D) {
    return gdn::supported(D) ? (size_t)gdn::kBackwardCtas * D * sizeof(float) : 0;
}

gdn_status gdn_qk_norm_rope_backward(const void *dq, const void *dk, const void *xq, const void *xk,
                                     gdn_dtype io_dtype, int64_t xq_stride, int64_t xk_stride,
                                     const float *wq, const float *wk, float eps, const int32_t *positions,
                                     int32_t axes, const int32_t *sections, const float *inv_freq,
                                     int32_t rot, int32_t interleaved, int64_t T, int32_t Hq, int32_t Hk,
                                     int32_t D, void *dxq, void *dxk, int64_t dxq_stride,
                                     int64_t dxk_stride, float *dwq, float *dwk, void *workspace,
                                     size_t workspace_bytes, void *stream) {
    GDN_TRACE("gdn_qk_norm_rope_backward");
    gdn::RopeArgs a{};
    if (gdn_status e = gdn::common(a, xq, xk, io_dtype, xq_stride, xk_stride, wq, wk, eps, positions, axes,
                                   sections, inv_freq, rot, interleaved, T, Hq, Hk, D))
        return e;
    if (T > 0 && (!dq || !dxq || (Hk > 0 && (!dk || !dxk)))) return GDN_ERR_INVALID_ARGUMENT;
    const int64_t esz = io_dtype == GDN_DTYPE_BF16 ? 2 : 4;
    if (dxq_stride < (int64_t)Hq * D || (Hk > 0 && dxk_stride < (int64_t)Hk * D)) return GDN_ERR_INVALID_ARGUMENT;
    if (dxq_stride > 0x3fffffff || (Hk > 0 && dxk_stride > 0x3fffffff)) return GDN_ERR_UNSUPPORTED;
    if ((dxq_stride * esz) % 16 || (Hk > 0 && (dxk_stride * esz) % 16)) return GDN_ERR_INVALID_ARGUMENT;
    const void *all[] = {dq, dk, xq, xk, wq, wk, positions, inv_freq, dxq, dxk, dwq, dwk, workspace};
    for (const void *p : all)
        if (p && !gdn::aligned16(p)) return GDN_ERR_INVALID_ARGUMENT;
    const void *ins[] = {dq, dk, xq, xk, wq, wk, positions, inv_freq};
    const void *outs[] = {dxq, dxk, dwq, dwk, workspace};
    for (int i = 0; i < 5; ++i) {
        for (const void *p : ins)
            if (outs[i] && outs[i] == p) return GDN_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (outs[i] && outs[i] == outs[j]) return GDN_ERR_INVALID_ARGUMENT;
    }
    const bool weights = dwq || dwk;
    if (weights && T > 0 &&
        (!workspace || workspace_bytes < gdn_qk_norm_rope_backward_workspace_bytes(D)))
        return GDN_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {  // no rows: the weights' gradients are zero
        for (float *p : {dwq, dwk})
            if (p && cudaMemsetAsync(p, 0, (size_t)D * sizeof(float), s) != cudaSuccess) return GDN_ERR_CUDA;
        return GDN_OK;
    }
    a.side[0].dz = dq;
    a.side[1].dz = dk;
    a.side[0].out = dxq;
    a.side[1].out = dxk;
    a.side[0].out_step = (uint32_t)(dxq_stride * esz);
    a.side[1].out_step = (uint32_t)(dxk_stride * esz);
    a.dw_part = weights ? static_cast<float *>(workspace) : nullptr;
    const cudaError_t e = io_dtype == GDN_DTYPE_BF16
                              ? gdn::dispatch<__nv_bfloat16>(a, D, true, dwq, dwk, s)
                              : gdn::dispatch<float>(a, D, true, dwq, dwk, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
