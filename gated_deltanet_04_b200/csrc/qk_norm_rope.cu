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
// Bound by HBM bandwidth: x is read once, z written once (backward: x and dz
// read, dx written).  A row is spread over D / 8 lanes with 8 elements each;
// rotation partners are another lane's same elements (rot % 16 == 0), one
// shuffle away.  A CTA takes kIter rows per lane group with all their loads in
// flight before the angles are computed.
#include "gdn_internal.cuh"
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
    int64_t T, rows;           // rows = T * H
};

// 8 consecutive elements of a row as fp32.
template <class E>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        v = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + i);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[j]));
            f[2 * j] = t.x;
            f[2 * j + 1] = t.y;
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, const float (&f)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
            u[j] = *reinterpret_cast<const uint32_t *>(&t);
        }
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + i) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        a = s[0];
        b = s[1];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, const float (&f)[8]) {
        float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        d[0] = make_float4(f[0], f[1], f[2], f[3]);
        d[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

template <int N>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int off = N / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// cos and sin of tokens t0 .. t0 + n - 1 into cs[token][rot/2] (cosines, then sines).
__device__ __forceinline__ void angles(const RopeArgs &a, int64_t t0, int n, float *cosines, float *sines) {
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const int64_t t = t0 + i / half;
        const int f = i % half;
        int axis = 0;
        while (axis < kMaxAxes - 1 && f >= a.last[axis]) ++axis;
        // whole turns removed in fp64: |turns| < 2^31 leaves 2^-22 of a turn at worst
        const double turns = (double)a.pos[axis * a.T + t] * ((double)a.inv_freq[f] * 0.15915494309189533577);
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        cosines[i] = c;
        sines[i] = s;
    }
}

__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Turns the lane's 8 elements (block l of the row) by its token's angles;
// sign = -1 turns them back.
template <int LPR>
__device__ __forceinline__ void rotate(float (&y)[8], int l, const float *c, const float *s, int rot,
                                       int interleaved, float sign) {
    const int hb = rot / 16;  // blocks per half of the rotated dimensions
    const bool in = l < 2 * hb;
    if (interleaved) {
        if (in) {
            const float4 c4 = *reinterpret_cast<const float4 *>(c + 4 * l);
            const float4 s4 = *reinterpret_cast<const float4 *>(s + 4 * l);
            const float cv[4] = {c4.x, c4.y, c4.z, c4.w}, sv[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float ss = sign * sv[j], p = y[2 * j], q = y[2 * j + 1];
                y[2 * j] = p * cv[j] - q * ss;
                y[2 * j + 1] = q * cv[j] + p * ss;
            }
        }
        return;
    }
    if (hb == 0) return;
    const bool lower = l < hb;
    const int lane = threadIdx.x & 31, src = in ? (lower ? lane + hb : lane - hb) : lane;
    const int b = in ? (lower ? l : l - hb) : 0;
    const float sg = lower ? -sign : sign;
    float cv[8], sv[8];
    load8(c + 8 * b, cv);
    load8(s + 8 * b, sv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float other = __shfl_sync(0xffffffffu, y[j], src);
        if (in) y[j] = y[j] * cv[j] + sg * other * sv[j];
    }
}

// A CTA's rows: `first` and the following ones, as tokens and heads.  The one
// 64-bit division is the CTA's; a row's place is 32-bit arithmetic from there.
struct Rows {
    int64_t t0;     // token of the first row
    uint32_t h0;    // its head
    uint32_t n;     // rows
    uint32_t n_tok;
    __device__ __forceinline__ Rows(const RopeArgs &a, int64_t first, int per) {
        t0 = first / a.H;
        h0 = (uint32_t)(first - t0 * a.H);
        n = (uint32_t)(a.rows - first < per ? a.rows - first : per);
        n_tok = (h0 + n - 1) / (uint32_t)a.H + 1;
    }
};
// Row r of them: its token (from t0), whether it is a key's, its elements' offset within the token.
template <int D>
struct Row {
    uint32_t tok;
    int z, off;
    __device__ __forceinline__ Row(const RopeArgs &a, const Rows &rows, uint32_t r, int l) {
        const uint32_t x = rows.h0 + r;
        tok = x / (uint32_t)a.H;
        const int h = (int)(x - tok * (uint32_t)a.H);
        z = h >= a.Hq;
        off = (h - (z ? a.Hq : 0)) * D + 8 * l;
    }
};

template <class E, int D, int kIter>
__global__ void __launch_bounds__(kThreads) gdn_qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
    extern __shared__ __align__(16) float smem[];
    constexpr int LPR = D / 8, GROUPS = kThreads / LPR;
    const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const Rows rows(a, (int64_t)blockIdx.x * (GROUPS * kIter), GROUPS * kIter);
    Vec8<E> x[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const uint32_t r = i * GROUPS + grp;
        if (r < rows.n) {
            const Row<D> w(a, rows, r, l);
            x[i].load(a.x[w.z], (rows.t0 + w.tok) * a.x_stride[w.z] + w.off);
        }
    }
    const int half = a.rot / 2;
    float *cosines = smem, *sines = smem + rows.n_tok * half;
    angles(a, rows.t0, (int)rows.n_tok, cosines, sines);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const uint32_t r = i * GROUPS + grp;
        const bool live = r < rows.n;  // every lane runs the shuffles
        const Row<D> w(a, rows, live ? r : 0, l);
        float y[8];
        if (live) {
            x[i].get(y);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = 0.f;
        }
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
        const float rms = rsqrtf(group_sum<LPR>(ss) * (1.f / D) + a.eps);
        const float *wt = a.w[w.z];
        if (wt) {
            float wv[8];
            load8(wt + 8 * l, wv);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= rms * wv[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= rms;
        }
        const int off = (int)w.tok * half;
        rotate<LPR>(y, l, cosines + off, sines + off, a.rot, a.interleaved, 1.f);
        if (live) Vec8<E>::store(a.out[w.z], (rows.t0 + w.tok) * a.out_stride[w.z] + w.off, y);
    }
}

// Persistent: CTA b takes row blocks b, b + grid, ...; each lane keeps its 8
// columns of both weight gradients in registers, summed over the CTA at the
// end and over the CTAs by a second kernel (a fixed order, no atomics).
template <class E, int D, int kIter>
__global__ void __launch_bounds__(kThreads)
    gdn_qk_norm_rope_backward_kernel(const __grid_constant__ RopeArgs a) {
    extern __shared__ __align__(16) float smem[];
    constexpr int LPR = D / 8, GROUPS = kThreads / LPR;
    const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const int half = a.rot / 2;
    float acc[2][8];
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[z][j] = 0.f;
    for (int64_t first = (int64_t)blockIdx.x * (GROUPS * kIter); first < a.rows;
         first += (int64_t)gridDim.x * (GROUPS * kIter)) {
        const Rows rows(a, first, GROUPS * kIter);
        Vec8<E> x[kIter], g[kIter];
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const uint32_t r = i * GROUPS + grp;
            if (r < rows.n) {
                const Row<D> w(a, rows, r, l);
                x[i].load(a.x[w.z], (rows.t0 + w.tok) * a.x_stride[w.z] + w.off);
                g[i].load(a.dz[w.z], (rows.t0 + w.tok) * a.dz_stride[w.z] + w.off);
            }
        }
        __syncthreads();  // the previous block's angles have been read
        float *cosines = smem, *sines = smem + rows.n_tok * half;
        angles(a, rows.t0, (int)rows.n_tok, cosines, sines);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const uint32_t r = i * GROUPS + grp;
            const bool live = r < rows.n;
            const Row<D> w(a, rows, live ? r : 0, l);
            float n[8], dy[8];
            if (live) {
                x[i].get(n);
                g[i].get(dy);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) n[j] = dy[j] = 0.f;
            }
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(n[j], n[j], ss);
            const float rms = rsqrtf(group_sum<LPR>(ss) * (1.f / D) + a.eps);
            const int off = (int)w.tok * half;
            rotate<LPR>(dy, l, cosines + off, sines + off, a.rot, a.interleaved, -1.f);
            float wv[8];
            if (a.w[w.z]) {
                load8(a.w[w.z] + 8 * l, wv);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) wv[j] = 1.f;
            }
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n[j] *= rms;
                const float dn = dy[j] * n[j];  // a dead row's is 0 times 0
                acc[0][j] += w.z ? 0.f : dn;
                acc[1][j] += w.z ? dn : 0.f;
                dy[j] *= wv[j];
                dot = fmaf(dy[j], n[j], dot);
            }
            dot = group_sum<LPR>(dot) * (1.f / D);
#pragma unroll
            for (int j = 0; j < 8; ++j) dy[j] = rms * (dy[j] - n[j] * dot);
            if (live) Vec8<E>::store(a.out[w.z], (rows.t0 + w.tok) * a.out_stride[w.z] + w.off, dy);
        }
    }
    if (!a.dw_part) return;
    // sum over the CTA's lane groups: [2][D] from GROUPS partials, in order
    __syncthreads();
#pragma unroll
    for (int z = 0; z < 2; ++z) {
#pragma unroll
        for (int j = 0; j < 8; ++j) smem[grp * D + 8 * l + j] = acc[z][j];
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

template <class E, int D>
cudaError_t launch_forward(const RopeArgs &a, cudaStream_t s) {
    constexpr int GROUPS = kThreads / (D / 8);
    // four rows per lane group once that still fills the GPU: their loads
    // overlap and the angles are shared; one row each below that (latency)
    const bool many = a.rows >= (int64_t)GROUPS * 4 * 592;
    const int iter = many ? 4 : 1;
    const int64_t blocks = (a.rows + GROUPS * iter - 1) / (GROUPS * iter);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const size_t smem = (size_t)tokens_of(GROUPS * iter, a.H) * a.rot * sizeof(float);
    auto *fn = many ? gdn_qk_norm_rope_kernel<E, D, 4> : gdn_qk_norm_rope_kernel<E, D, 1>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    fn<<<(unsigned)blocks, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <class E, int D>
cudaError_t launch_backward(const RopeArgs &a, float *dwq, float *dwk, cudaStream_t s) {
    constexpr int GROUPS = kThreads / (D / 8), kIter = sizeof(E) == 2 ? 4 : 2;
    const int64_t blocks = (a.rows + GROUPS * kIter - 1) / (GROUPS * kIter);
    const int ctas = (int)(blocks < kBackwardCtas ? blocks : kBackwardCtas);
    size_t smem = (size_t)tokens_of(GROUPS * kIter, a.H) * a.rot * sizeof(float);
    if (smem < (size_t)GROUPS * D * sizeof(float)) smem = (size_t)GROUPS * D * sizeof(float);
    auto *fn = gdn_qk_norm_rope_backward_kernel<E, D, kIter>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    fn<<<ctas, kThreads, smem, s>>>(a);
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
    if (!supported(D) || rot % 16 != 0) return GDN_ERR_UNSUPPORTED;
    a.x[0] = xq; a.x[1] = xk;
    a.w[0] = wq; a.w[1] = wk;
    a.x_stride[0] = xq_stride; a.x_stride[1] = xk_stride;
    a.pos = positions; a.inv_freq = inv_freq; a.eps = eps;
    a.Hq = Hq; a.H = Hq + Hk; a.rot = rot; a.interleaved = interleaved;
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
