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
constexpr int kBackwardCtas = 592;  // persistent grid of the backward pass (4 per SM of 148)

struct RopeArgs {
    const void *x[2];          // q, k inputs
    const void *dz[2];         // backward: gradients of the outputs
    void *out[2];              // outputs, or the gradients of x
    const float *w[2];         // [D] or null (ones)
    float *dw_part;            // backward: [CTAs][2][D] or null
    int64_t x_stride[2], out_stride[2], dz_stride[2];  // elements per token
    const int32_t *pos;        // [axes][T]
    const float *inv_freq;     // [rot / 2]
    int32_t last[kMaxAxes];    // frequency i belongs to the first axis with i < last[axis]
    float eps;
    int32_t Hq, H, rot, interleaved;
    uint32_t inv_h, inv_half;  // ceil(2^32 / H) (H > 1), ceil(2^32 / (rot / 2))
    int32_t blocks;            // blocks of kIter rows per lane group that share their angles
    int64_t T, rows;           // rows = T * H
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
    __device__ __forceinline__ void load(const void *p, int64_t i, const Pieces &c) {
        a = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + i + c.p0);
        b = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + i + c.p1);
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
    static __device__ __forceinline__ void store(void *p, int64_t i, const Pieces &c, const float2 (&f)[4]) {
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p) + i + c.p0) = make_uint2(narrow(f[0]), narrow(f[1]));
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p) + i + c.p1) = make_uint2(narrow(f[2]), narrow(f[3]));
    }
};
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void *p, int64_t i, const Pieces &c) {
        a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + c.p0);
        b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + c.p1);
    }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
        f[0] = make_float2(a.x, a.y);
        f[1] = make_float2(a.z, a.w);
        f[2] = make_float2(b.x, b.y);
        f[3] = make_float2(b.z, b.w);
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, const Pieces &c, const float2 (&f)[4]) {
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + i + c.p0) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + i + c.p1) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
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

// A CTA's rows: `first` and the following ones, as tokens and heads.
struct Rows {
    int64_t t0;     // token of the first row
    uint32_t h0;    // its head
    uint32_t n;     // rows
    uint32_t n_tok;
    __device__ __forceinline__ Rows(const RopeArgs &a, int64_t first, int per) {
        // (a 64-bit division only where 32 bits do not hold the row)
        t0 = a.rows >> 32 ? first / a.H : (int64_t)((uint32_t)first / (uint32_t)a.H);
        h0 = (uint32_t)(first - t0 * a.H);
        n = (uint32_t)(a.rows - first < per ? a.rows - first : per);
        n_tok = (h0 + n - 1) / (uint32_t)a.H + 1;
    }
};
// Row r of them: its token (from t0), whether it is a key's, its offset within the token.
template <int D>
struct Row {
    uint32_t tok;
    int z, off;
    __device__ __forceinline__ Row(const RopeArgs &a, const Rows &rows, uint32_t r) {
        const uint32_t x = rows.h0 + r;  // x H < 2^32: the product with ceil(2^32 / H) divides exactly
        tok = a.H == 1 ? x : __umulhi(x, a.inv_h);
        const int h = (int)(x - tok * (uint32_t)a.H);
        z = h >= a.Hq;
        off = (h - (z ? a.Hq : 0)) * D;
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
    const Pieces c(l, a.rot, a.interleaved);
    const Rows rows(a, (int64_t)blockIdx.x * (kBlock * a.blocks), kBlock * a.blocks);
    Vec8<E> next[kIter];
    auto load = [&](uint32_t r0) {
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const uint32_t r = r0 + i * GROUPS;
            if (r < rows.n) {
                const Row<D> w(a, rows, r);
                next[i].load(a.x[w.z], (rows.t0 + w.tok) * a.x_stride[w.z] + w.off, c);
            }
        }
    };
    load(grp);
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
            const Row<D> w(a, rows, live ? r : 0);
            float2 y[4];
            x[i].get(y);
            const float2 rms = splat(rsqrtf(group_sum<LPR>(dot8(y, y)) * (1.f / D) + a.eps));
            if (a.w[w.z]) {
                float2 wv[4];
                load_pieces(a.w[w.z], c, wv);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = fmul2(y[j], fmul2(rms, wv[j]));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = fmul2(y[j], rms);
            }
            const int off = (int)w.tok * half;
            rotate(y, c, cosines + off, sines + off, a.interleaved, 1.f);
            if (live) Vec8<E>::store(a.out[w.z], (rows.t0 + w.tok) * a.out_stride[w.z] + w.off, c, y);
        }
    }
}

// Persistent: CTA b takes the rows of blocks b, b + grid, ... (each a.blocks
// blocks, as above); each lane keeps its 8 columns of both weight gradients in
// registers, summed over the CTA at the end and over the CTAs by a second kernel
// (a fixed order, no atomics).
template <class E, int D, int kIter>
__global__ void __launch_bounds__(kThreads, sizeof(E) == 2 ? 3 : 2)
    gdn_qk_norm_rope_backward_kernel(const __grid_constant__ RopeArgs a) {
    extern __shared__ __align__(16) float smem[];
    constexpr int LPR = D / 8, GROUPS = kThreads / LPR, kBlock = GROUPS * kIter;
    const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const Pieces c(l, a.rot, a.interleaved);
    const int half = a.rot / 2;
    float2 acc[2][4];
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[z][j] = splat(0.f);
    const int64_t per = (int64_t)kBlock * a.blocks;
    for (int64_t first = blockIdx.x * per; first < a.rows; first += gridDim.x * per) {
        const Rows rows(a, first, (int)per);
        Vec8<E> next_x[kIter], next_g[kIter];
        auto load = [&](uint32_t r0) {
#pragma unroll
            for (int i = 0; i < kIter; ++i) {
                const uint32_t r = r0 + i * GROUPS;
                if (r < rows.n) {
                    const Row<D> w(a, rows, r);
                    next_x[i].load(a.x[w.z], (rows.t0 + w.tok) * a.x_stride[w.z] + w.off, c);
                    next_g[i].load(a.dz[w.z], (rows.t0 + w.tok) * a.dz_stride[w.z] + w.off, c);
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
                const Row<D> w(a, rows, live ? r : 0);
                float2 n[4], dy[4];
                x[i].get(n);
                g[i].get(dy);
                const float rms = rsqrtf(group_sum<LPR>(dot8(n, n)) * (1.f / D) + a.eps);
                const int off = (int)w.tok * half;
                rotate(dy, c, cosines + off, sines + off, a.interleaved, -1.f);
                float2 wv[4];
                if (a.w[w.z]) {
                    load_pieces(a.w[w.z], c, wv);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) wv[j] = splat(1.f);
                }
                // selected, not multiplied by 0 or 1: a key's infinity stays the key's
                const bool to_q = live && !w.z, to_k = live && w.z;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    n[j] = fmul2(n[j], splat(rms));
                    const float2 dn = fmul2(dy[j], n[j]);
                    acc[0][j].x += to_q ? dn.x : 0.f;
                    acc[0][j].y += to_q ? dn.y : 0.f;
                    acc[1][j].x += to_k ? dn.x : 0.f;
                    acc[1][j].y += to_k ? dn.y : 0.f;
                    dy[j] = fmul2(dy[j], wv[j]);
                }
                const float2 dot = splat(-group_sum<LPR>(dot8(dy, n)) * (1.f / D));
#pragma unroll
                for (int j = 0; j < 4; ++j) dy[j] = fmul2(ffma2(n[j], dot, dy[j]), splat(rms));
                if (live) Vec8<E>::store(a.out[w.z], (rows.t0 + w.tok) * a.out_stride[w.z] + w.off, c, dy);
            }
        }
    }
    if (!a.dw_part) return;
    // sum over the CTA's lane groups: [2][D] from GROUPS partials, in order
    __syncthreads();
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        float *mine = smem + grp * D;
        *reinterpret_cast<float4 *>(mine + c.p0) = make_float4(acc[z][0].x, acc[z][0].y, acc[z][1].x, acc[z][1].y);
        *reinterpret_cast<float4 *>(mine + c.p1) = make_float4(acc[z][2].x, acc[z][2].y, acc[z][3].x, acc[z][3].y);
        __syncthreads();
        for (int d = threadIdx.x; d < D; d += kThreads) {
            float s = 0.f;
            for (int q = 0; q < GROUPS; ++q) s += smem[q * D + d];
            a.dw_part[((int64_t)blockIdx.x * 2 + z) * D + d] = s;
        }
        __syncthreads();
    }
}

// dw[z][d] = sum over CTAs of part[cta][z][d]: a warp per column.
__global__ void gdn_qk_norm_dw_kernel(const float *part, int ctas, int D, float *dwq, float *dwk) {
    const int col = (blockIdx.x * blockDim.x + threadIdx.x) / 32, lane = threadIdx.x & 31;
    if (col >= 2 * D) return;
    float s = 0.f;
    for (int c = lane; c < ctas; c += 32) s += part[(int64_t)c * 2 * D + col];
    s = group_sum<32>(s);
    float *dst = col < D ? dwq : dwk;
    if (lane == 0 && dst) dst[col < D ? col : col - D] = s;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool supported(int32_t D) { return D == 16 || D == 32 || D == 64 || D == 128 || D == 256; }

// Tokens a block of `rows` consecutive rows can touch.
int64_t tokens_of(int64_t rows, int32_t H) { return rows / H + 2; }

// Blocks of `block` rows per CTA, so that their angles are computed once: as many
// (up to `most`) as keep `ctas` CTAs busy and the angles within 40 KB.
int blocks_per_cta(const RopeArgs &a, int64_t block, int64_t ctas, int most) {
    int n = 1;
    while (n < most && a.rows >= block * 2 * n * ctas &&
           tokens_of(block * 2 * n, a.H) * a.rot * (int64_t)sizeof(float) <= 40 * 1024)
        n *= 2;
    return n;
}

template <class E, int D>
cudaError_t launch_forward(RopeArgs a, cudaStream_t s) {
    constexpr int GROUPS = kThreads / (D / 8);
    // two rows per lane group at a time once that still fills the GPU, one below (latency)
    const bool many = a.rows >= (int64_t)GROUPS * 2 * 592;
    const int block = GROUPS * (many ? 2 : 1);
    a.blocks = many ? blocks_per_cta(a, block, 592, 8) : 1;
    const int64_t per = (int64_t)block * a.blocks, ctas = (a.rows + per - 1) / per;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    const size_t smem = (size_t)tokens_of(per, a.H) * a.rot * sizeof(float);
    auto *fn = many ? gdn_qk_norm_rope_kernel<E, D, 2> : gdn_qk_norm_rope_kernel<E, D, 1>;
    fn<<<(unsigned)ctas, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <class E, int D>
cudaError_t launch_backward(RopeArgs a, float *dwq, float *dwk, cudaStream_t s) {
    constexpr int GROUPS = kThreads / (D / 8), kIter = 2;
    const int block = GROUPS * kIter;
    a.blocks = blocks_per_cta(a, block, kBackwardCtas, 8);
    const int64_t per = (int64_t)block * a.blocks, want = (a.rows + per - 1) / per;
    const int ctas = (int)(want < kBackwardCtas ? want : kBackwardCtas);
    size_t smem = (size_t)tokens_of(per, a.H) * a.rot * sizeof(float);
    if (smem < (size_t)GROUPS * D * sizeof(float)) smem = (size_t)GROUPS * D * sizeof(float);
    gdn_qk_norm_rope_backward_kernel<E, D, kIter><<<ctas, kThreads, smem, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.dw_part) return e;
    gdn_qk_norm_dw_kernel<<<(2 * D * 32 + 255) / 256, 256, 0, s>>>(a.dw_part, ctas, D, dwq, dwk);
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
    if ((xq_stride * esz) % 16 || (Hk > 0 && (xk_stride * esz) % 16)) return GDN_ERR_INVALID_ARGUMENT;
    if (!supported(D) || rot % 16 != 0 || Hq > 32768 - Hk) return GDN_ERR_UNSUPPORTED;
    a.x[0] = xq; a.x[1] = xk;
    a.w[0] = wq; a.w[1] = wk;
    a.x_stride[0] = xq_stride; a.x_stride[1] = xk_stride;
    a.pos = positions; a.inv_freq = inv_freq; a.eps = eps;
    a.Hq = Hq; a.H = Hq + Hk;
    auto inverse = [](uint32_t n) { return (uint32_t)((((uint64_t)1 << 32) + n - 1) / n); };
    a.inv_h = inverse((uint32_t)a.H);
    a.inv_half = rot > 0 ? inverse((uint32_t)rot / 2) : 0;
    a.rot = rot; a.interleaved = interleaved;
    a.T = T; a.rows = T * (int64_t)(Hq + Hk);
    return a.rows > ((int64_t)1 << 33) ? GDN_ERR_UNSUPPORTED : GDN_OK;  // the grid's x dimension
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
    a.out[0] = q; a.out[1] = k;
    a.out_stride[0] = (int64_t)Hq * D; a.out_stride[1] = (int64_t)Hk * D;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = io_dtype == GDN_DTYPE_BF16
                              ? gdn::dispatch<__nv_bfloat16>(a, D, false, nullptr, nullptr, s)
                              : gdn::dispatch<float>(a, D, false, nullptr, nullptr, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_qk_norm_rope_backward_workspace_bytes(int32_t D) {
    return gdn::supported(D) ? (size_t)gdn::kBackwardCtas * 2 * D * sizeof(float) : 0;
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
    a.dz[0] = dq; a.dz[1] = dk;
    a.dz_stride[0] = (int64_t)Hq * D; a.dz_stride[1] = (int64_t)Hk * D;
    a.out[0] = dxq; a.out[1] = dxk;
    a.out_stride[0] = dxq_stride; a.out_stride[1] = dxk_stride;
    a.dw_part = weights ? static_cast<float *>(workspace) : nullptr;
    const cudaError_t e = io_dtype == GDN_DTYPE_BF16
                              ? gdn::dispatch<__nv_bfloat16>(a, D, true, dwq, dwk, s)
                              : gdn::dispatch<float>(a, D, true, dwq, dwk, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
