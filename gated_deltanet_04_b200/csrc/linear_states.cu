// Chunk states of linear attention on tensor cores (StatePass, linear_tc.cuh).
//
// One CTA walks the chunks of one (segment, head).  The state is held in
// registers, fp32, 64 values of a row per thread; each chunk's sum of outer
// products is one fresh tensor-core accumulator added to it in fp32 (the tensor
// core's own accumulation over thousands of chunks would truncate, and with a
// slow decay the loss would add up).
//
// Precision: y enters as it is (bf16); x times its decay weight is split into
// two bf16 parts, hi + lo, which keeps 16 bits of it (2^-17 relative on
// average): two MMA passes instead of one, so that the fp32 states are good to
// a few 1e-6.
//
// Per chunk: TMA brings x and y; the threads turn x in place into hi and write
// lo beside it; the MMAs of chunk c run while the threads add chunk c - 1's
// result to the state and store the image of the state that enters c.  Two
// stages of (y, hi, lo) and the image take 224 KB of shared memory.
// Bound: HBM (64 KB in, 32 KB image out per chunk and head, y shared by the
// heads of a group through L2) against 2 x 4.2 MFLOP on the tensor core.
#include "linear_tc.cuh"

namespace gdn {
namespace linear {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t OFF_STAGE = 3 * kTile;  // y, x / hi, lo
constexpr uint32_t OFF_IMAGE = 2 * OFF_STAGE;
constexpr uint32_t OFF_MISC = OFF_IMAGE + kTile;

struct Misc {
    uint64_t full[2], done[2];
    uint32_t tmem;
};
constexpr uint32_t kSmem = OFF_MISC + sizeof(Misc) + 1024;
static_assert(kSmem <= 232448, "shared memory of an SM");

// kDump: the pass proper (images, final state); otherwise the segments' sums.
template <bool kDump>
__global__ void __launch_bounds__(kThreads, 1)
    gdn_linear_states_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y,
                             StatePass p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc *ms = reinterpret_cast<Misc *>(sm + OFF_MISC);
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, half = warp >> 2;
    const int row = quad * 32 + lane;  // row of M, its columns 64 half ..

    const int h = blockIdx.x % p.H;
    const int64_t slot = blockIdx.x / p.H;
    const int64_t seg_len = p.seg ? p.seg_chunks * kC : (p.T > 0 ? p.T : 1);
    Span sp;
    if (!find_span(p.cu, p.N, p.T, seg_len, slot, p.err, sp)) return;
    const bool last = p.reverse ? sp.s == 0 : sp.s == sp.count - 1;  // in the pass's order
    if (!kDump && last) return;  // nothing starts from its sum
    const int hy = h / (p.H / p.Hy);
    const int nch = (int)((sp.t1 - sp.t0 + kC - 1) / kC);
    const float l2 = p.log_decay[h] * kLog2e;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ms->full[s], 1);
            mbar_init(&ms->done[s], 1);
        }
        fence_mbarrier_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_y);
    }
    if (warp == 0) {
        tmem_alloc(&ms->tmem, 256);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = ms->tmem;
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16) + 64 * half;

    auto chunk_at = [&](int it) { return p.reverse ? nch - 1 - it : it; };
    auto issue = [&](int it) {  // thread 0
        uint8_t *st = sm + (it & 1) * OFF_STAGE;
        const int64_t t = sp.t0 + (int64_t)chunk_at(it) * kC;
        mbar_arrive_expect_tx(&ms->full[it & 1], 2 * kTile);
        load_tile(st + kTile, &tm_x, &ms->full[it & 1], h, t);
        load_tile(st, &tm_y, &ms->full[it & 1], hy, t);
    };
    int issued = 0;  // thread 0's count
    if (tid == 0)
        for (; issued < nch && issued < 2; ++issued) issue(issued);

    float S[64];
    const int64_t st = kDump ? state_index(p.map, sp.n) : 0;
    if (kDump && st < 0 && tid == 0 && h == 0) raise_error(p.err, GDN_ERR_BAD_SLOT);
    {
        const float *src = nullptr;
        if (kDump && p.seg) src = p.seg + ((slot * p.H + h) * kD + row) * (int64_t)kD + 64 * half;
        else if (kDump && p.m0 && st >= 0 && !state_fresh(p.map, sp.n))
            src = p.m0 + ((st * p.H + h) * kD + row) * (int64_t)kD + 64 * half;
#pragma unroll
        for (int x = 0; x < 64; x += 4) {
            const float4 f = src ? *reinterpret_cast<const float4 *>(src + x) : make_float4(0.f, 0.f, 0.f, 0.f);
            S[x] = f.x; S[x + 1] = f.y; S[x + 2] = f.z; S[x + 3] = f.w;
        }
    }
    // weight of row j of a chunk of L tokens (0 past its end)
    auto weight = [&](int j, int L) {
        if (j >= L) return 0.f;
        return p.reverse ? p.x_scale * exp2f(l2 * (float)(j + 1)) : exp2f(l2 * (float)(L - 1 - j));
    };
    float wfull[4];  // this thread converts rows tid / 8 + 32 i
#pragma unroll
    for (int i = 0; i < 4; ++i) wfull[i] = weight((tid >> 3) + 32 * i, kC);
    const float dec_full = exp2f(l2 * (float)kC);

    bool timed_out = false;
    // S <- lam^L S + chunk it's sum, once its MMAs are done
    auto finish = [&](int it) {
        if (!mbar_wait_bounded(&ms->done[it & 1], (it >> 1) & 1, kWaitLimit)) timed_out = true;
        tc_fence_after_sync();
        const int64_t left = sp.t1 - (sp.t0 + (int64_t)chunk_at(it) * kC);
        const float dec = left < kC ? exp2f(l2 * (float)left) : dec_full;
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
            float d[32];
            tmem_ld32(trow + 128 * (it & 1) + c, d);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) S[c + x] = fmaf(dec, S[c + x], d[x]);
        }
    };
    int it = 0;
#pragma unroll 1
    for (; it < nch; ++it) {
        uint8_t *stg = sm + (it & 1) * OFF_STAGE;
        const int c = chunk_at(it);
        const int64_t left = sp.t1 - (sp.t0 + (int64_t)c * kC);
        const int L = left < kC ? (int)left : kC;
        if (!mbar_wait_bounded(&ms->full[it & 1], (it >> 1) & 1, kWaitLimit)) timed_out = true;
        // 16-byte pieces: rows tid / 8 + 32 i of both column halves
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = (tid >> 3) + 32 * i;
            const float w = L == kC ? wfull[i] : weight(j, L);
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                uint8_t *at = stg + kTile + sub * kSub + j * 128 + (tid & 7) * 16;
                uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
                if (j < L) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(at);
                    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                    uint32_t oh[4], ol[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&in[q]));
                        const float a = f.x * w, b = f.y * w;
                        oh[q] = pack_bf16(a, b);
                        const float2 r = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&oh[q]));
                        ol[q] = pack_bf16(a - r.x, b - r.y);
                    }
                    hi = make_uint4(oh[0], oh[1], oh[2], oh[3]);
                    lo = make_uint4(ol[0], ol[1], ol[2], ol[3]);
                } else {
                    // rows of the next sequence: y too, or its NaN would reach this sum
                    *reinterpret_cast<uint4 *>(at - kTile) = hi;
                }
                *reinterpret_cast<uint4 *>(at) = hi;
                *reinterpret_cast<uint4 *>(at + kTile) = lo;
            }
        }
        fence_proxy_async_smem();
        if (kDump && tid == 0) bulk_wait_read_all();  // the image buffer is free again
        tc_fence_before_sync();
        if (__syncthreads_or(timed_out ? 1 : 0)) break;
        tc_fence_after_sync();
        if (tid == 0) {
            const uint32_t y = sbase + (it & 1) * OFF_STAGE, d = tmem + 128 * (it & 1);
            mma_mm(d, y + kTile, y, false);
            mma_mm(d, y + 2 * kTile, y, true);
            mma_commit(&ms->done[it & 1]);
        }
        if (it > 0) {
            finish(it - 1);
            if (tid == 0 && issued < nch) {  // its stage is free
                issue(issued);
                ++issued;
            }
        }
        if (kDump) {
#pragma unroll
            for (int x = 0; x < 64; x += 8) {
                const uint4 v = make_uint4(pack_bf16(S[x], S[x + 1]), pack_bf16(S[x + 2], S[x + 3]),
                                           pack_bf16(S[x + 4], S[x + 5]), pack_bf16(S[x + 6], S[x + 7]));
                *reinterpret_cast<uint4 *>(sm + OFF_IMAGE + half * kSub + sw128(row, 2 * x)) = v;
            }
            fence_proxy_async_smem();
            __syncthreads();
            if (tid == 0) {
                const int64_t cs = slot_base(p.cu, sp.n, kC) + (sp.t0 - (p.cu ? p.cu[sp.n] : 0)) / kC + c;
                bulk_store(p.dump + (cs * p.H + h) * (int64_t)kTile, sm + OFF_IMAGE, kTile);
                bulk_commit();
            }
        }
    }
    const bool ok = it == nch;
    if (ok && nch > 0) finish(nch - 1);
    if (!ok || timed_out) {
        if (tid == 0) raise_error(p.err, GDN_ERR_TIMEOUT);
        // a bounded chance for the MMAs and tile loads in flight to land
        for (int s = 0; s < 2; ++s) {
            const int k = it - 1 - ((it - 1 - s) & 1);  // the last chunk whose MMAs used barrier s
            if (it > 0 && k >= 0) mbar_wait_bounded(&ms->done[s], (k >> 1) & 1, kWaitLimit);
        }
        if (tid == 0)
            for (int k = it; k < issued; ++k) mbar_wait_bounded(&ms->full[k & 1], (k >> 1) & 1, kWaitLimit);
    } else {
        float *dst = kDump ? (last && p.mT && st >= 0 ? p.mT + (st * p.H + h) * (int64_t)(kD * kD) : nullptr)
                           : p.seg + (slot * p.H + h) * (int64_t)(kD * kD);
        if (dst) {
            dst += (int64_t)row * kD + 64 * half;
#pragma unroll
            for (int x = 0; x < 64; x += 4)
                *reinterpret_cast<float4 *>(dst + x) = make_float4(S[x], S[x + 1], S[x + 2], S[x + 3]);
        }
    }
    if (kDump && tid == 0) bulk_wait_all();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, 256);
}

template <bool kDump>
cudaError_t launch(const CUtensorMap &mx, const CUtensorMap &my, const StatePass &p, cudaStream_t s) {
    const int64_t len = p.seg ? p.seg_chunks * kC : (p.T > 0 ? p.T : 1);
    const int64_t blocks = slots_of(p.T, p.N, len) * p.H;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(gdn_linear_states_kernel<kDump>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    gdn_linear_states_kernel<kDump><<<(unsigned)blocks, kThreads, kSmem, s>>>(mx, my, p);
    return cudaGetLastError();
}

}  // namespace

int device_sms() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

// Segments when the (sequence, head) units alone would leave SMs idle: as many
// as let whole waves of 148 CTAs share the chunks, up to four waves for long
// sequences (a shorter last wave), none under 4 chunks.
int64_t state_seg_chunks(int32_t N, int64_t T, int32_t H) {
    const int64_t chunks = T / kC + 1, units = (int64_t)N * H;
    if (units <= 0 || T <= 0) return 0;
    int64_t waves = chunks * H / (148 * 16);
    waves = waves < 1 ? 1 : waves > 4 ? 4 : waves;
    const int64_t want = 148 * waves / H;  // segments, were all of one sequence's length
    if (want <= 1) return 0;
    int64_t len = (chunks + want - 1) / want;
    len = len < 4 ? 4 : len;
    return len < chunks ? len : 0;
}

size_t state_seg_bytes(int32_t N, int64_t T, int32_t H) {
    const int64_t c = state_seg_chunks(N, T, H);
    return c ? (size_t)slots_of(T, N, c * kC) * H * kD * kD * 4 : 0;
}

size_t state_dump_bytes(int32_t N, int64_t T, int32_t H) { return (size_t)slots_of(T, N, kC) * H * kTile; }

cudaError_t launch_states(const StatePass &p, cudaStream_t s) {
    CUtensorMap mx, my;
    const int64_t Tm = p.T > 0 ? p.T : 1;
    if (!make_tile_map_bf16_128(&mx, p.x, Tm, p.H, kC) || !make_tile_map_bf16_128(&my, p.y, Tm, p.Hy, kC))
        return cudaErrorInvalidValue;
    if (p.seg) {
        cudaError_t e = launch<false>(mx, my, p, s);
        if (e != cudaSuccess) return e;
        Pass scan{};
        scan.H = p.H; scan.Da = kD; scan.Dc = kD; scan.log_decay = p.log_decay; scan.reverse = p.reverse;
        scan.m0 = p.m0; scan.map = p.map; scan.cu = p.cu; scan.N = p.N; scan.T = p.T; scan.err = p.err;
        scan.seg = p.seg; scan.seg_len = p.seg_chunks * kC;
        e = launch_scan(scan, s);
        if (e != cudaSuccess) return e;
    }
    return launch<true>(mx, my, p, s);
}

}  // namespace linear
}  // namespace gdn
