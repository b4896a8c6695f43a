// Linear attention passes (linear.cuh) token by token in fp32 on CUDA cores.
//
// Serves the head sizes and dtypes the tensor-core chunked kernels do not.
// Rows of M are independent given a and b, so a CTA owns some rows of one
// (segment, head), each row spread over Da / 16 lanes with 16 columns per lane
// in registers.  Per token a lane does 3 FMAs per column (decay, update,
// read-out) and one shuffle reduction of the read-out.  Token inputs come
// through shared memory, kTokBlock at a time, the next block's loads in flight
// while one is computed.
#include "linear.cuh"
#include "sm100.cuh"

namespace gdn {
namespace linear {
namespace {

using sm100::ffma2;
using sm100::fmul2;

constexpr int kTokBlock = 16;
constexpr int kThreads = 128;

template <int DA>
struct Shape {
    static constexpr int LPR = DA / 16;               // lanes per row
    static constexpr int RPT = DA == 16 ? 1 : 2;      // rows per thread
    static constexpr int ROWS = RPT * kThreads / LPR; // rows per CTA
};

__device__ __forceinline__ float4 load4(const void *p, int64_t idx, gdn_dtype dt) {
    if (dt == GDN_DTYPE_BF16) {
        const uint2 raw = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + idx);
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&raw.x));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&raw.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + idx);
}

template <int DA, bool kOut, bool kRev>
__global__ void __launch_bounds__(kThreads)
    gdn_linear_recurrent_kernel(Pass p, int row_blocks) {
    using S = Shape<DA>;
    constexpr int LPR = S::LPR, RPT = S::RPT, ROWS = S::ROWS;
    __shared__ __align__(16) float as_[kTokBlock][DA];
    __shared__ __align__(16) float bs[kTokBlock][DA];
    __shared__ __align__(16) float cs[kTokBlock][ROWS];
    __shared__ float os[kTokBlock][ROWS];

    const int tid = threadIdx.x;
    const int rb = blockIdx.x % row_blocks;
    const int h = (blockIdx.x / row_blocks) % p.H;
    const int64_t slot = blockIdx.x / (row_blocks * p.H);
    if (tid == kThreads - 1) check_range(p.cu, p.N, p.T, slot, p.err);
    Span sp;
    if (!find_span(p.cu, p.N, p.T, p.seg ? p.seg_len : (p.T > 0 ? p.T : 1), slot, p.err, sp)) return;
    const bool last = kRev ? sp.s == 0 : sp.s == sp.count - 1;  // in the pass's order
    if (!kOut && last) return;  // nothing starts from its sum
    const int row0 = rb * ROWS;
    const int l = tid % LPR;
    int rows[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) rows[r] = tid / LPR + r * (kThreads / LPR);

    const int64_t seg_off = (slot * p.H + h) * (int64_t)p.Dc * DA;
    const int64_t st = kOut ? state_index(p.map, sp.n) : 0;
    if (kOut && st < 0 && tid == 0 && rb == 0 && h == 0) raise_error(p.err, GDN_ERR_BAD_SLOT);
    const int64_t st_off = (st * p.H + h) * (int64_t)p.Dc * DA;

    // columns m*4*LPR + 4*l + (0, 1), (2, 3) of row rows[r]: pairs, for two multiply-adds an
    // instruction
    float2 M[RPT][8];
    const bool from_seg = kOut && p.seg && sp.count > 1;
    const bool from_m0 = kOut && !from_seg && p.m0 && st >= 0 && !state_fresh(p.map, sp.n);
    const float *src = from_seg ? p.seg + seg_off : from_m0 ? p.m0 + st_off : nullptr;
    const bool across = from_m0 && p.m0_transposed;  // M[i][d] is at [d][i]
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int i = row0 + rows[r], d = m * 4 * LPR + 4 * l;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (src && i < p.Dc) {
                if (across)
                    v = make_float4(src[(int64_t)d * p.Dc + i], src[(int64_t)(d + 1) * p.Dc + i],
                                    src[(int64_t)(d + 2) * p.Dc + i], src[(int64_t)(d + 3) * p.Dc + i]);
                else
                    v = *reinterpret_cast<const float4 *>(src + (int64_t)i * DA + d);
            }
            M[r][2 * m] = make_float2(v.x, v.y);
            M[r][2 * m + 1] = make_float2(v.z, v.w);
        }
    const Decay decay(p.log_decay[h]);
    const int64_t len = sp.t1 - sp.t0;
    const int64_t stride_a = (int64_t)p.Ha * DA, stride_b = (int64_t)p.Hb * DA,
                  stride_c = (int64_t)p.Hc * p.Dc, stride_o = (int64_t)p.Hout * p.Dc;
    const int64_t off_a = (int64_t)(h / (p.H / p.Ha)) * DA, off_b = (int64_t)(h / (p.H / p.Hb)) * DA,
                  off_c = (int64_t)(h / (p.H / p.Hc)) * p.Dc + row0,
                  off_o = (int64_t)(h / (p.H / p.Hout)) * p.Dc + row0;
    auto token = [&](int64_t pos) { return kRev ? sp.t1 - 1 - pos : sp.t0 + pos; };

    constexpr int VA = kTokBlock * DA / 4, NA = (VA + kThreads - 1) / kThreads;
    constexpr int VC = kTokBlock * ROWS / 4, NC = (VC + kThreads - 1) / kThreads;
    float4 ra[NA], rbv[NA], rc[NC];
    auto fetch = [&](int64_t pos) {
#pragma unroll
        for (int x = 0; x < NA; ++x) {
            const int idx = tid + x * kThreads, tt = idx / (DA / 4), c4 = idx % (DA / 4);
            ra[x] = rbv[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (idx < VA && pos + tt < len) {
                const int64_t t = token(pos + tt);
                if (kOut) ra[x] = load4(p.a, t * stride_a + off_a + 4 * c4, p.dtype);
                rbv[x] = load4(p.b, t * stride_b + off_b + 4 * c4, p.dtype);
            }
        }
#pragma unroll
        for (int x = 0; x < NC; ++x) {
            const int idx = tid + x * kThreads, tt = idx / (ROWS / 4), c4 = idx % (ROWS / 4);
            rc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (idx < VC && pos + tt < len && row0 + 4 * c4 < p.Dc)
                rc[x] = load4(p.c, token(pos + tt) * stride_c + off_c + 4 * c4, p.dtype);
        }
    };
    if (len > 0) fetch(0);
    for (int64_t pos = 0; pos < len; pos += kTokBlock) {
        const int nt = len - pos < kTokBlock ? (int)(len - pos) : kTokBlock;
#pragma unroll
        for (int x = 0; x < NA; ++x) {
            const int idx = tid + x * kThreads;
            if (idx < VA) {
                if (kOut) reinterpret_cast<float4 *>(&as_[0][0])[idx] = ra[x];
                reinterpret_cast<float4 *>(&bs[0][0])[idx] = rbv[x];
            }
        }
#pragma unroll
        for (int x = 0; x < NC; ++x) {
            const int idx = tid + x * kThreads;
            if (idx < VC) {
                const float4 v = rc[x];
                reinterpret_cast<float4 *>(&cs[0][0])[idx] =
                    make_float4(v.x * p.c_scale, v.y * p.c_scale, v.z * p.c_scale, v.w * p.c_scale);
            }
        }
        __syncthreads();
        if (pos + kTokBlock < len) fetch(pos + kTokBlock);
        auto compute = [&](auto slow) {  // a uniform choice, made once per block of tokens
            constexpr bool kSlow = decltype(slow)::value;
            // one token: the read-outs' partial sums of this lane's columns
            auto token_step = [&](int tt, float (&acc)[RPT]) {
                float2 cv[RPT], part[RPT][4];
#pragma unroll
                for (int r = 0; r < RPT; ++r) cv[r] = make_float2(cs[tt][rows[r]], cs[tt][rows[r]]);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float4 b4 = *reinterpret_cast<const float4 *>(&bs[tt][m * 4 * LPR + 4 * l]);
                    float4 a4;
                    if (kOut) a4 = *reinterpret_cast<const float4 *>(&as_[tt][m * 4 * LPR + 4 * l]);
                    const float2 bv[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
                    const float2 av[2] = {make_float2(a4.x, a4.y), make_float2(a4.z, a4.w)};
#pragma unroll
                    for (int r = 0; r < RPT; ++r) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float2 &x = M[r][2 * m + e];
                            if (!kRev) x = decay.times<kSlow>(x);
                            x = ffma2(cv[r], bv[e], x);
                            if (kOut) part[r][m] = e ? ffma2(x, av[e], part[r][m]) : fmul2(x, av[e]);
                            if (kRev) x = decay.times<kSlow>(x);
                        }
                    }
                }
                if (kOut) {
#pragma unroll
                    for (int r = 0; r < RPT; ++r)
                        acc[r] = ((part[r][0].x + part[r][0].y) + (part[r][1].x + part[r][1].y)) +
                                 ((part[r][2].x + part[r][2].y) + (part[r][3].x + part[r][3].y));
                }
            };
            // sums over the row's lanes, staged by the first of them
            auto finish = [&](int tt, float (&acc)[RPT]) {
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
#pragma unroll
                    for (int off = LPR / 2; off > 0; off >>= 1)
                        acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], off);
                    if (l == 0) os[tt][rows[r]] = acc[r] * p.out_scale;
                }
            };
            // four tokens at a time: their sums' latencies overlap
            int tt = 0;
            for (; tt + 4 <= nt; tt += 4) {
                float acc[4][RPT];
#pragma unroll
                for (int i = 0; i < 4; ++i) token_step(tt + i, acc[i]);
                if (kOut) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) finish(tt + i, acc[i]);
                }
            }
            for (; tt < nt; ++tt) {
                float acc[RPT];
                token_step(tt, acc);
                if (kOut) finish(tt, acc);
            }
        };
        if (decay.slow) compute(std::true_type{});
        else compute(std::false_type{});
        __syncthreads();  // the block's inputs are consumed and its outputs staged
        if (kOut) {
            for (int idx = tid; idx < nt * ROWS; idx += kThreads) {
                const int tt = idx / ROWS, i = idx % ROWS;
                if (row0 + i < p.Dc)
                    store_io(p.out, token(pos + tt) * stride_o + off_o + i, os[tt][i], p.out_dtype);
            }
        }
    }
    float *dst = kOut ? (last && p.mT && st >= 0 ? p.mT + st_off : nullptr) : p.seg + seg_off;
    if (dst) {
#pragma unroll
        for (int r = 0; r < RPT; ++r)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int i = row0 + rows[r], d = m * 4 * LPR + 4 * l;
                if (i < p.Dc)
                    *reinterpret_cast<float4 *>(dst + (int64_t)i * DA + d) =
                        make_float4(M[r][2 * m].x, M[r][2 * m].y, M[r][2 * m + 1].x, M[r][2 * m + 1].y);
            }
    }
}

// One thread per four elements of a (sequence, head) state: walks the
// sequence's segments in the pass's order, replacing each segment's sum by the
// state that enters it.
template <int kAhead>
__global__ void gdn_linear_scan_kernel(const __grid_constant__ Pass p0, const __grid_constant__ Pass p1) {
    const Pass &p = blockIdx.z ? p1 : p0;
    next_may_start();
    prior_done();
    const int n = blockIdx.x / p.H, h = blockIdx.x % p.H;
    const int per = p.Dc * p.Da;
    const int x = 4 * (int)(blockIdx.y * blockDim.x + threadIdx.x);
    if (x >= per) return;
    int64_t t0, t1;
    if (!seq_range(p.cu, n, p.N, p.T, p.err, t0, t1)) return;
    const int64_t count = t1 > t0 ? (t1 - t0 + p.seg_len - 1) / p.seg_len : 1;
    if (count == 1) return;  // the pass itself starts from the entering state
    const int64_t base = slot_base(p.cu, n, p.seg_len);
    const float g = p.log_decay[h];
    const Decay whole(g * (float)p.seg_len), tail(g * (float)(t1 - t0 - (count - 1) * p.seg_len));
    float4 cur = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t st = state_index(p.map, n);
    if (p.m0 && st >= 0 && !state_fresh(p.map, n)) {
        const float *src = p.m0 + (st * p.H + h) * (int64_t)per;
        if (p.m0_transposed) {
            const int i = x / p.Da, d = x % p.Da;
            cur = make_float4(src[(int64_t)d * p.Dc + i], src[(int64_t)(d + 1) * p.Dc + i],
                              src[(int64_t)(d + 2) * p.Dc + i], src[(int64_t)(d + 3) * p.Dc + i]);
        } else {
            cur = *reinterpret_cast<const float4 *>(src + x);
        }
    }
    auto seg = [&](int64_t j) { return p.reverse ? count - 1 - j : j; };
    auto at = [&](int64_t j) {
        return reinterpret_cast<float4 *>(p.seg + ((base + seg(j)) * p.H + h) * (int64_t)per + x);
    };
    // the sums of kAhead segments, and those of the next ones in flight meanwhile
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 own[kAhead], next[kAhead];
    auto load = [&](int64_t j0) {  // (the last segment's sum is not there: nothing starts from it)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) next[i] = j0 + i + 1 < count ? *at(j0 + i) : zero;
    };
    load(0);
    for (int64_t j0 = 0; j0 < count; j0 += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) own[i] = next[i];
        if (j0 + kAhead < count) load(j0 + kAhead);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t j = j0 + i;
            if (j >= count) break;
            *at(j) = cur;
            const Decay d = seg(j) == count - 1 ? tail : whole;
            auto add = [&](auto slow) {
                constexpr bool kSlow = decltype(slow)::value;
                const float2 lo = d.plus<kSlow>(make_float2(cur.x, cur.y), make_float2(own[i].x, own[i].y));
                const float2 hi = d.plus<kSlow>(make_float2(cur.z, cur.w), make_float2(own[i].z, own[i].w));
                cur = make_float4(lo.x, lo.y, hi.x, hi.y);
            };
            if (d.slow) add(std::true_type{});
            else add(std::false_type{});
        }
    }
}

__global__ void gdn_linear_group_sum_kernel(const float *src, void *dst, gdn_dtype dt, int64_t total,
                                            int32_t G, int32_t D) {
    for (int64_t i = 4 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x); i < total;
         i += 4 * (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / D, d = i % D;  // row = token * Hout + group
        const float *p = src + row * G * D + d;
        float4 s = *reinterpret_cast<const float4 *>(p);
        for (int g = 1; g < G; ++g) {
            const float4 x = *reinterpret_cast<const float4 *>(p + (int64_t)g * D);
            s.x += x.x;
            s.y += x.y;
            s.z += x.z;
            s.w += x.w;
        }
        if (dt == GDN_DTYPE_BF16) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
            uint2 raw;
            raw.x = *reinterpret_cast<const uint32_t *>(&lo);
            raw.y = *reinterpret_cast<const uint32_t *>(&hi);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(dst) + i) = raw;
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(dst) + i) = s;
        }
    }
}

template <int DA>
cudaError_t launch(const Pass &p, int phase, cudaStream_t s) {
    const int row_blocks = (p.Dc + Shape<DA>::ROWS - 1) / Shape<DA>::ROWS;
    const int64_t slots = slots_of(p.T, p.N, p.seg ? p.seg_len : (p.T > 0 ? p.T : 1));
    const int64_t blocks = slots * p.H * row_blocks;
    if (blocks <= 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(kThreads);
    if (phase == 1) {
        if (p.reverse) gdn_linear_recurrent_kernel<DA, false, true><<<grid, block, 0, s>>>(p, row_blocks);
        else gdn_linear_recurrent_kernel<DA, false, false><<<grid, block, 0, s>>>(p, row_blocks);
    } else {
        if (p.reverse) gdn_linear_recurrent_kernel<DA, true, true><<<grid, block, 0, s>>>(p, row_blocks);
        else gdn_linear_recurrent_kernel<DA, true, false><<<grid, block, 0, s>>>(p, row_blocks);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_recurrent(const Pass &p, int phase, cudaStream_t s) {
    switch (p.Da) {
        case 16: return launch<16>(p, phase, s);
        case 32: return launch<32>(p, phase, s);
        case 64: return launch<64>(p, phase, s);
        case 128: return launch<128>(p, phase, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_scan(const Pass *passes, int count, cudaStream_t s) {
    const Pass &p = passes[0];
    const int64_t units = (int64_t)p.N * p.H;
    if (units <= 0) return cudaSuccess;
    if (units > 0x7fffffffLL) return cudaErrorInvalidValue;
    const int per = p.Dc * p.Da / 4, threads = per < 256 ? per : 256;
    // the longest sequence's segments: with four at most (the tensor-core prefill of one
    // sequence) fewer registers are in the way of the next kernel's start (4,096 tokens, 48
    // heads: 106.5 us and 109.3); with many, more loads in flight (64 segments: 13 us and 21)
    return launch_after(p.T <= 4 * p.seg_len ? gdn_linear_scan_kernel<4> : gdn_linear_scan_kernel<8>, true,
                        dim3((unsigned)units, (unsigned)((per + threads - 1) / threads), count), threads, 0, s, p,
                        passes[count - 1]);
}

// Enough segments for about eight of the 128-thread CTAs on each of 148 SMs,
// none shorter than 64 tokens, or 32 where a state is 64 x 64 or smaller: a token is
// 0.17 us of latency in a pass, a segment costs its state's traffic and its step of the
// scan.  (1,024 tokens, 4 heads: gradients at 64 x 64 84 us in segments of 32 and 103 of
// 64, prefill at 128 x 128 48 and 43.)
int64_t recurrent_seg_len(int32_t N, int64_t T, int32_t H, int32_t Da, int32_t Dc) {
    const int rows = Da == 16 ? 128 : 2 * kThreads / (Da / 16);
    const int64_t ctas = (int64_t)N * H * ((Dc + rows - 1) / rows);
    if (ctas <= 0 || T <= 0) return 0;
    const int64_t want = (148 * 8 + ctas - 1) / ctas;
    if (want <= 1) return 0;
    int64_t len = (T + want - 1) / want;
    const int64_t least = Da * Dc > 64 * 64 ? 64 : 32;
    len = len < least ? least : (len + kTokBlock - 1) / kTokBlock * kTokBlock;
    return len < T ? len : 0;
}

cudaError_t launch_group_sum(const float *src, void *dst, gdn_dtype dt, int64_t T, int32_t H,
                             int32_t Hout, int32_t D, cudaStream_t s) {
    const int64_t total = T * Hout * D;
    if (total <= 0) return cudaSuccess;
    const int64_t want = (total / 4 + 255) / 256;
    gdn_linear_group_sum_kernel<<<(unsigned)(want < 4736 ? want : 4736), 256, 0, s>>>(src, dst, dt, total,
                                                                                    H / Hout, D);
    return cudaGetLastError();
}

}  // namespace linear
}  // namespace gdn
