// One-token update of linear attention with a decay per head, in place on the
// state: S <- lam S + v k^T, o = scale S q per (sequence, v-head).
//
// Bound by HBM bandwidth on the state, 8 Dv Dk bytes read and written per unit;
// each row is loaded, updated, reduced against q and stored by the same lanes.
// Row i of Dk fp32 values is spread over Dk / 4 lanes as float4.
//
// Dk = 128, the workload's: a warp takes kRows rows of a unit at once, all their
// loads in flight, and sums their dot products together by recursive halving
// (kRows shuffles and one, instead of 5 kRows).  16 rows a warp when there are
// units enough to fill the GPU so, 4 when there are few (latency).
// Other Dk: a CTA of 8 warps serves one unit, with kRows row groups in flight.
#include "linear.cuh"

namespace gdn {
namespace linear {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 8;

__device__ __forceinline__ float4 load4(const void *p, int64_t idx, gdn_dtype dt) {
    if (dt == GDN_DTYPE_BF16) {
        const uint2 raw = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + idx);
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&raw.x));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&raw.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + idx);
}

template <int DK>
__global__ void __launch_bounds__(kWarps * 32) gdn_linear_decode_kernel(DecodeStep d) {
    constexpr int LPR = DK / 4, RP = 32 / LPR, STRIDE = kWarps * RP;
    const int h = blockIdx.x % d.Hv, n = blockIdx.x / d.Hv, j = h / (d.Hv / d.Hqk);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR, l = lane % LPR;
    const int64_t slot = state_index(d.map, n);
    if (slot < 0) {  // a bad slot index: this unit writes nothing
        if (threadIdx.x == 0) raise_error(d.err, GDN_ERR_BAD_SLOT);
        return;
    }
    const bool fresh = state_fresh(d.map, n);
    const int64_t qk = ((int64_t)n * d.Hqk + j) * DK + 4 * l;
    const float4 kk = load4(d.k, qk, d.dtype), qq = load4(d.q, qk, d.dtype);
    const Decay decay(d.log_decay[h]);
    auto times = [&](float x) { return decay.slow ? decay.times<true>(x) : decay.times<false>(x); };
    float *st = d.state + (slot * d.Hv + h) * (int64_t)d.Dv * DK;
    const int64_t vo = (int64_t)blockIdx.x * d.Dv;
    for (int w0 = warp * RP; w0 < d.Dv; w0 += STRIDE * kRows) {  // w0 is warp-uniform
        float4 row[kRows];
        float vi[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int i = w0 + sub + r * STRIDE;
            row[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            vi[r] = 0.f;
            if (i < d.Dv) {
                if (!fresh) row[r] = __ldcs(reinterpret_cast<const float4 *>(st + (int64_t)i * DK) + l);
                vi[r] = load_io(d.v, vo + i, d.dtype);
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int i = w0 + sub + r * STRIDE;
            float4 s = row[r];
            s.x = fmaf(vi[r], kk.x, times(s.x));
            s.y = fmaf(vi[r], kk.y, times(s.y));
            s.z = fmaf(vi[r], kk.z, times(s.z));
            s.w = fmaf(vi[r], kk.w, times(s.w));
            float dot = s.x * qq.x + s.y * qq.y + s.z * qq.z + s.w * qq.w;
#pragma unroll
            for (int off = LPR / 2; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
            if (i < d.Dv) {
                __stcs(reinterpret_cast<float4 *>(st + (int64_t)i * DK) + l, s);
                if (l == 0) store_io(d.o, vo + i, dot * d.scale, d.dtype);
            }
        }
    }
}

// Sums each of R values over the warp: lane L returns the sum of value L / (32 / R).
template <int R>
__device__ __forceinline__ float transposed_sum(float (&v)[R], int lane) {
#pragma unroll
    for (int n = R, off = 16; n > 1; n /= 2, off /= 2) {
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float send = up ? v[i] : v[i + n / 2], keep = up ? v[i + n / 2] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
#pragma unroll
    for (int off = 16 / R; off > 0; off /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    return v[0];
}

template <int R>
__global__ void __launch_bounds__(kWarps * 32) gdn_linear_decode128_kernel(DecodeStep d, int blocks) {
    const int unit = blockIdx.x / blocks, h = unit % d.Hv, n = unit / d.Hv, j = h / (d.Hv / d.Hqk);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i0 = ((blockIdx.x % blocks) * kWarps + warp) * R;  // this warp's rows
    const int64_t slot = state_index(d.map, n);
    if (slot < 0) {  // a bad slot index: this unit writes nothing
        if (threadIdx.x == 0) raise_error(d.err, GDN_ERR_BAD_SLOT);
        return;
    }
    if (i0 >= d.Dv) return;
    const bool fresh = state_fresh(d.map, n);
    float4 *st = reinterpret_cast<float4 *>(d.state + ((slot * d.Hv + h) * (int64_t)d.Dv + i0) * 128) + lane;
    const int rows = d.Dv - i0;  // those of them that exist (R or more: all)
    float4 s[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        s[r] = !fresh && r < rows ? __ldcs(st + 32 * r) : make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t qk = ((int64_t)n * d.Hqk + j) * 128 + 4 * lane, vo = (int64_t)unit * d.Dv + i0;
    const float4 kk = load4(d.k, qk, d.dtype), qq = load4(d.q, qk, d.dtype);
    const float vl = lane < R && lane < rows ? load_io(d.v, vo + lane, d.dtype) : 0.f;
    const Decay decay(d.log_decay[h]);
    auto times = [&](float x) { return decay.slow ? decay.times<true>(x) : decay.times<false>(x); };
    float dot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float v = __shfl_sync(0xffffffffu, vl, r);
        s[r].x = fmaf(v, kk.x, times(s[r].x));
        s[r].y = fmaf(v, kk.y, times(s[r].y));
        s[r].z = fmaf(v, kk.z, times(s[r].z));
        s[r].w = fmaf(v, kk.w, times(s[r].w));
        if (r < rows) __stcs(st + 32 * r, s[r]);
        dot[r] = s[r].x * qq.x + s[r].y * qq.y + s[r].z * qq.z + s[r].w * qq.w;
    }
    const float o = transposed_sum<R>(dot, lane);
    const int r = lane / (32 / R);
    if (lane % (32 / R) == 0 && r < rows) store_io(d.o, vo + r, o * d.scale, d.dtype);
}

template <int R>
cudaError_t launch128(const DecodeStep &d, int64_t units, cudaStream_t s) {
    const int blocks = (d.Dv + kWarps * R - 1) / (kWarps * R);
    if (units * blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    gdn_linear_decode128_kernel<R><<<(unsigned)(units * blocks), kWarps * 32, 0, s>>>(d, blocks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode(const DecodeStep &d, cudaStream_t s) {
    const int64_t units = (int64_t)d.N * d.Hv;
    if (units <= 0) return cudaSuccess;
    if (units > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)units), block(kWarps * 32);
    switch (d.Dk) {
        case 16: gdn_linear_decode_kernel<16><<<grid, block, 0, s>>>(d); break;
        case 32: gdn_linear_decode_kernel<32><<<grid, block, 0, s>>>(d); break;
        case 64: gdn_linear_decode_kernel<64><<<grid, block, 0, s>>>(d); break;
        case 128: return units * ((d.Dv + 127) / 128) >= 296 ? launch128<16>(d, units, s) : launch128<4>(d, units, s);
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

}  // namespace linear
}  // namespace gdn
