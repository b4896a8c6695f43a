// Chunk states of linear attention on tensor cores (StatePass, linear_tc.cuh).
//
// One CTA walks the chunks of one (segment, head).  The fp32 state stays in
// tensor memory; each chunk's sum of outer products is one fresh tensor-core
// accumulator added to it by fp32 FMAs (the tensor core's own accumulation over
// thousands of chunks would truncate, and with a slow decay the loss would add
// up).
//
// Precision: y enters as it is (bf16); x times its decay weight is split into
// bf16 parts, hi + mid + lo, which together keep fp32's 24 bits: three MMA
// passes, wherever the sum goes into an fp32 state.  Where only bf16 images
// come of it (a segment that does not end its sequence), hi + mid do.
//
// Shared memory bandwidth bounds this kernel (128 B a clock; the products alone
// read 64 KB per part, chunk and head), so x does not pass through it on its
// way in: the converting warps load it from global memory, a stage ahead.
//
// Roles, on stages of 64 tokens: a producer warp loads y by TMA into a ring; 16
// warps write x's parts into two buffers in turn; an MMA warp sums a chunk's
// stages into one of two accumulators; 8 warps add it to the state and store the
// image of the state that enters the next chunk.
// Bound: HBM (64 KB in, 32 KB image out per chunk and head, y shared by the
// heads of a group through L2) against two or three products of 4.2 MFLOP.
#include "linear_tc.cuh"

namespace gdn {
namespace linear {
namespace {

constexpr int kRows = 64;                    // tokens per stage
constexpr uint32_t kHalf = kRows * 128;      // 64 rows x 64 columns
constexpr uint32_t kPart = 2 * kHalf;        // 64 x 128 bf16
constexpr int kRing = 6;                     // stages of y
constexpr int kStateWarps = 8, kConvWarps = 16;
constexpr int kStateThreads = kStateWarps * 32, kConvThreads = kConvWarps * 32;
constexpr int kThreads = kStateThreads + kConvThreads + 64;
constexpr uint32_t TM_S = 256;               // tensor memory: two sums, the state
constexpr uint32_t OFF_PARTS = kRing * kPart;           // [2][hi, mid, lo]
constexpr uint32_t OFF_IMAGE = OFF_PARTS + 6 * kPart;
constexpr uint32_t OFF_MISC = OFF_IMAGE + kTile;

struct Misc {
    uint64_t raw_full[kRing], raw_empty[kRing], part_full[2], part_empty[2], sum_full[2], sum_empty[2], drain;
    uint32_t tmem;
    volatile int32_t abort;
};
constexpr uint32_t kSmem = OFF_MISC + sizeof(Misc) + 1024;
static_assert(kSmem <= 232448, "shared memory of an SM");

// The chunks of a segment in the pass's order: tokens t0 .. t0 + len - 1.
struct Walk {
    int64_t t0;
    int32_t len, nch;
    bool reverse;
    __device__ __forceinline__ int chunk(int it) const { return reverse ? nch - 1 - it : it; }
    __device__ __forceinline__ int length(int it) const { return min(len - chunk(it) * kC, kC); }
};

__device__ void produce(const CUtensorMap &tm_y, const Walk &w, int hy, uint8_t *sm, Misc *ms, int32_t *err) {
    uint32_t r = 0;  // stages so far
    for (int it = 0; it < w.nch; ++it) {
        const int L = w.length(it);
        for (int j0 = 0; j0 < L; j0 += kRows, ++r) {
            const int b = r % kRing;
            if (r >= kRing && !role_wait(&ms->raw_empty[b], (r / kRing - 1) & 1, &ms->abort, err)) {
                // given up: let the loads in flight land before the CTA ends
                for (uint32_t x = r - kRing; x < r; ++x)
                    mbar_wait_bounded(&ms->raw_full[x % kRing], (x / kRing) & 1, kWaitLimit);
                return;
            }
            uint8_t *y = sm + b * kPart;
            const int32_t t = (int32_t)w.t0 + w.chunk(it) * kC + j0;
            mbar_arrive_expect_tx(&ms->raw_full[b], kPart);
            tma_load_3d(y, &tm_y, &ms->raw_full[b], 0, hy, t);
            tma_load_3d(y + kHalf, &tm_y, &ms->raw_full[b], 64, hy, t);
        }
    }
}

// A weight in three bf16 parts (24 bits), each twice in a word.
struct Weight {
    uint32_t h, m, l;
};
__device__ __forceinline__ uint32_t twice_bf16(float x) { return pack_bf16(x, x); }
__device__ __forceinline__ Weight split_weight(float w) {
    Weight f;
    f.h = twice_bf16(w);
    const float r = w - unpack_bf16(f.h).x;
    f.m = twice_bf16(r);
    f.l = twice_bf16(r - unpack_bf16(f.m).x);
    return f;
}

// Packed bf16 pairs: fused multiply-add, product, difference, one rounding each.
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    return fma2(a, b, 0x80008000u);  // - 0: keeps the sign of a zero product
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) { return fma2(b, 0xbf80bf80u, a); }  // a - b

// x w = hi + mid + lo, stage after stage into the two parts buffers in turn, in
// packed bf16 arithmetic (fused multiply-adds, one rounding each): hi = x wh
// rounded; x wh - hi is exact (16 bits less the upper 8), so mid = x wm + (x wh -
// hi) is rounded once, and lo takes what mid's rounding left and x wl.
// x: head h's row of token 0, `stride` elements from token to token.
template <int kParts>
__device__ void convert(const Walk &w, const __nv_bfloat16 *x, int64_t stride, float l2, float x_scale, uint8_t *sm,
                        Misc *ms, int tid, int32_t *err) {
    const int r0 = tid >> 4, col = (tid & 15) * 8;  // rows r0 and r0 + 32 of a stage, 8 columns from col
    const uint32_t at = (col >> 6) * kHalf + sw128(r0, (col & 63) * 2);  // row r0 + 32: 4096 further
    // weight of row j of a chunk of L tokens (0 past its end)
    auto weight = [&](int j, int L) {
        if (j >= L) return 0.f;
        return w.reverse ? x_scale * exp2f(l2 * (float)(j + 1)) : exp2f(l2 * (float)(L - 1 - j));
    };
    // a thread's share of a stage: rows r0 and r0 + 32; weights of a whole chunk's stages
    const Weight whole[2][2] = {{split_weight(weight(r0, kC)), split_weight(weight(r0 + 32, kC))},
                                {split_weight(weight(r0 + 64, kC)), split_weight(weight(r0 + 96, kC))}};
    uint4 v[2][2];  // x of the next chunk's stages
    auto load = [&](int it, int s) {
        if (it >= w.nch) return;
        const int c = w.chunk(it), left = w.len - c * kC - s * kRows - r0;
        const __nv_bfloat16 *src = x + (w.t0 + c * kC + s * kRows + r0) * stride + col;
        v[s][0] = left > 0 ? __ldg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0u, 0u, 0u, 0u);
        v[s][1] = left > 32 ? __ldg(reinterpret_cast<const uint4 *>(src + 32 * stride)) : make_uint4(0u, 0u, 0u, 0u);
    };
    uint32_t r = 0;
    auto piece = [&](const uint4 &x4, const Weight &f, uint8_t *dst) {
        const uint32_t in[4] = {x4.x, x4.y, x4.z, x4.w};
        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            hi[q] = mul2(in[q], f.h);
            const uint32_t rest = fma2(in[q], f.h, hi[q] ^ 0x80008000u);
            mid[q] = fma2(in[q], f.m, rest);
            if (kParts == 3) lo[q] = fma2(in[q], f.l, fma2(in[q], f.m, sub2(rest, mid[q])));
        }
        *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(dst + kPart) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
        if (kParts == 3) *reinterpret_cast<uint4 *>(dst + 2 * kPart) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    };
    load(0, 0);
    load(0, 1);
    for (int it = 0; it < w.nch; ++it) {
        const int L = w.length(it);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (s * kRows >= L) {  // a short chunk's second stage
                load(it + 1, s);
                continue;
            }
            const int buf = r & 1, left = L - s * kRows;
            if (r >= 2 && !role_wait(&ms->part_empty[buf], ((r >> 1) - 1) & 1, &ms->abort, err)) return;
            uint8_t *dst = sm + OFF_PARTS + buf * 3 * kPart + at;
            if (L == kC) {
                piece(v[s][0], whole[s][0], dst);
                piece(v[s][1], whole[s][1], dst + 4096);
            } else {
                piece(v[s][0], split_weight(weight(s * kRows + r0, L)), dst);
                piece(v[s][1], split_weight(weight(s * kRows + r0 + 32, L)), dst + 4096);
            }
            load(it + 1, s);
            if (left < kRows) {  // rows of the next sequence: 0 times their NaN would reach this sum
                const int b = r % kRing;
                if (!role_wait(&ms->raw_full[b], (r / kRing) & 1, &ms->abort, err)) return;
                for (int k = tid; k < (kRows - left) * 16; k += kConvThreads)
                    *reinterpret_cast<uint4 *>(sm + b * kPart + (k & 1) * kHalf + left * 128 + (k >> 1) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            warp_arrive(&ms->part_full[buf]);
            ++r;
        }
    }
}

// Sums a chunk's stages: D = (hi + mid + lo)^T y, both operands MN-major.
template <int kParts>
__device__ void multiply(const Walk &w, uint32_t sbase, uint32_t tmem, Misc *ms, int32_t *err) {
    uint32_t r = 0, b = 0, lap = 0;  // stages so far; the ring's stage and lap
    const uint64_t y0 = desc_m(sbase, kHalf), x0 = desc_m(sbase + OFF_PARTS, kHalf);
    bool ok = true;
    for (int it = 0; ok && it < w.nch; ++it) {
        const int L = w.length(it);
        const uint32_t d = tmem + 128 * (it & 1);
        if (it >= 2 && !(ok = role_wait(&ms->sum_empty[it & 1], ((it >> 1) - 1) & 1, &ms->abort, err))) break;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (s * kRows >= L) break;
            const uint32_t buf = r & 1;
            if (!(ok = role_wait(&ms->raw_full[b], lap & 1, &ms->abort, err) &&
                       role_wait(&ms->part_full[buf], (r >> 1) & 1, &ms->abort, err)))
                break;
            tc_fence_after_sync();
            const uint64_t y = y0 + b * (kPart >> 4), x = x0 + buf * (3 * kPart >> 4);
#pragma unroll
            for (int k = 0; k < kParts; ++k)
#pragma unroll
                for (int ks = 0; ks < kRows / 16; ++ks)
                    mma_f16_ss(d, step_m(x + (k * kPart >> 4), ks), step_m(y, ks), IDESC_MM, s || k || ks);
            mma_commit(&ms->raw_empty[b]);
            mma_commit(&ms->part_empty[buf]);
            ++r;
            if (++b == kRing) {
                b = 0;
                ++lap;
            }
        }
        if (ok) mma_commit(&ms->sum_full[it & 1]);
    }
    if (ok) return;
    // given up: let the MMAs in flight finish before tensor memory is freed
    mma_commit(&ms->drain);
    mbar_wait_bounded(&ms->drain, 0, kWaitLimit);
}

__device__ __forceinline__ void state_barrier() {
    asm volatile("bar.sync 1, %0;" ::"n"(kStateThreads) : "memory");
}

// kDump: the pass proper (images, final state); otherwise the segments' sums.
template <bool kDump>
__global__ void __launch_bounds__(kThreads, 1)
    gdn_linear_states_kernel(const __grid_constant__ CUtensorMap tm_y, StatePass p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc *ms = reinterpret_cast<Misc *>(sm + OFF_MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int h = blockIdx.x % p.H;
    const int64_t slot = blockIdx.x / p.H;
    const int64_t seg_len = p.seg ? p.seg_chunks * kC : (p.T > 0 ? p.T : 1);
    Span sp;
    if (!find_span(p.cu, p.N, p.T, seg_len, slot, p.err, sp)) return;
    const bool last = p.reverse ? sp.s == 0 : sp.s == sp.count - 1;  // in the pass's order
    if (!kDump && last) return;  // nothing starts from its sum
    const int hy = h / (p.H / p.Hy);
    const int32_t len = (int32_t)(sp.t1 - sp.t0);
    const Walk w{sp.t0, len, (len + kC - 1) / kC, p.reverse};
    const float l2 = p.log_decay[h] * kLog2e;
    const bool exact = !kDump || (last && p.mT);  // its sum goes into an fp32 state

    if (tid == 0) {
        for (int b = 0; b < kRing; ++b) {
            mbar_init(&ms->raw_full[b], 1);
            mbar_init(&ms->raw_empty[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ms->part_full[b], kConvWarps);
            mbar_init(&ms->part_empty[b], 1);
            mbar_init(&ms->sum_full[b], 1);
            mbar_init(&ms->sum_empty[b], kStateWarps);
        }
        mbar_init(&ms->drain, 1);
        ms->abort = 0;
        fence_mbarrier_init();
    }
    if (warp == 0) {
        tmem_alloc(&ms->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = ms->tmem;

    if (warp >= kStateWarps) {
        const int cw = warp - kStateWarps;
        if (cw < kConvWarps) {
            const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(p.x) + (int64_t)h * kD;
            if (exact) convert<3>(w, x, (int64_t)p.H * kD, l2, p.x_scale, sm, ms, tid - kStateThreads, p.err);
            else convert<2>(w, x, (int64_t)p.H * kD, l2, p.x_scale, sm, ms, tid - kStateThreads, p.err);
        } else if (cw == kConvWarps) {
            if (lane == 0) produce(tm_y, w, hy, sm, ms, p.err);
        } else if (lane == 0) {
            if (exact) multiply<3>(w, smem_u32(sm), tmem, ms, p.err);
            else multiply<2>(w, smem_u32(sm), tmem, ms, p.err);
        }
    } else {
        const int quad = warp & 3, half = warp >> 2, row = quad * 32 + lane;  // columns 64 half .. of row
        const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16) + 64 * half;
        const int64_t st = kDump ? state_index(p.map, sp.n) : 0;
        if (kDump && st < 0 && tid == 0 && h == 0) raise_error(p.err, GDN_ERR_BAD_SLOT);
        const int64_t at = (int64_t)row * kD + 64 * half;  // within a state
        uint8_t *image = sm + OFF_IMAGE + half * kSub;
        // columns c .. c + 15 of this thread's half row of the image
        auto draw = [&](int c, const float *v) {  // 16 of them
#pragma unroll
            for (int x = 0; x < 16; x += 8)
                *reinterpret_cast<uint4 *>(image + sw128(row, 2 * (c + x))) =
                    make_uint4(pack_bf16(v[x], v[x + 1]), pack_bf16(v[x + 2], v[x + 3]),
                               pack_bf16(v[x + 4], v[x + 5]), pack_bf16(v[x + 6], v[x + 7]));
        };
        const int64_t chunk0 = kDump ? slot_base(p.cu, sp.n, kC) + sp.s * (seg_len / kC) : 0;
        auto store_image = [&](int it) {  // the state entering chunk it; all state warps call
            fence_proxy_async_smem();
            state_barrier();
            if (tid == 0) {
                bulk_store(p.dump + ((chunk0 + w.chunk(it)) * p.H + h) * (int64_t)kTile, sm + OFF_IMAGE, kTile);
                bulk_commit();
            }
        };
        const float *src = nullptr;
        if (kDump && p.seg) src = p.seg + (slot * p.H + h) * (int64_t)(kD * kD) + at;
        else if (kDump && p.m0 && st >= 0 && !state_fresh(p.map, sp.n))
            src = p.m0 + (st * p.H + h) * (int64_t)(kD * kD) + at;
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
            float v[16];
#pragma unroll
            for (int x = 0; x < 16; x += 4) {
                const float4 f = src ? *reinterpret_cast<const float4 *>(src + c + x) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[x] = f.x; v[x + 1] = f.y; v[x + 2] = f.z; v[x + 3] = f.w;
            }
            tmem_st16(trow + TM_S + c, v);
            if (kDump && w.nch > 0) draw(c, v);
        }
        tmem_wait_st();
        if (kDump && w.nch > 0) store_image(0);
        const float dec_full = exp2f(l2 * (float)kC);
        bool ok = true;
        for (int it = 0; it < w.nch; ++it) {
            // every warp goes on after a wait given up, so that the barriers stay whole
            if (ok) ok = role_wait(&ms->sum_full[it & 1], (it >> 1) & 1, &ms->abort, p.err);
            tc_fence_after_sync();
            const bool more = kDump && it + 1 < w.nch;
            if (more) {
                if (tid == 0) bulk_wait_read_all();  // the image buffer is free again
                state_barrier();
            }
            const int L = w.length(it);
            const float dec = L < kC ? exp2f(l2 * (float)L) : dec_full;
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
                float v[16], d[16];
                tmem_ld16(trow + TM_S + c, v);
                tmem_ld16(trow + 128 * (it & 1) + c, d);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 16; ++x) v[x] = fmaf(dec, v[x], d[x]);
                tmem_st16(trow + TM_S + c, v);
                if (more) draw(c, v);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            warp_arrive(&ms->sum_empty[it & 1]);
            if (more) store_image(it + 1);
        }
        float *dst = kDump ? (last && p.mT && st >= 0 ? p.mT + (st * p.H + h) * (int64_t)(kD * kD) : nullptr)
                           : p.seg + (slot * p.H + h) * (int64_t)(kD * kD);
        if (ok && dst) {
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                float v[32];
                tmem_ld32(trow + TM_S + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 32; x += 4)
                    *reinterpret_cast<float4 *>(dst + at + c + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
            }
        }
        if (kDump && tid == 0) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <bool kDump>
cudaError_t launch(const CUtensorMap &my, const StatePass &p, cudaStream_t s) {
    const int64_t len = p.seg ? p.seg_chunks * kC : (p.T > 0 ? p.T : 1);
    const int64_t blocks = slots_of(p.T, p.N, len) * p.H;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(gdn_linear_states_kernel<kDump>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    gdn_linear_states_kernel<kDump><<<(unsigned)blocks, kThreads, kSmem, s>>>(my, p);
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
    CUtensorMap my;
    const int64_t Tm = p.T > 0 ? p.T : 1;
    if (!make_tile_map_bf16_128(&my, p.y, Tm, p.Hy, kRows)) return cudaErrorInvalidValue;
    if (p.seg) {
        cudaError_t e = launch<false>(my, p, s);
        if (e != cudaSuccess) return e;
        Pass scan{};
        scan.H = p.H; scan.Da = kD; scan.Dc = kD; scan.log_decay = p.log_decay; scan.reverse = p.reverse;
        scan.m0 = p.m0; scan.map = p.map; scan.cu = p.cu; scan.N = p.N; scan.T = p.T; scan.err = p.err;
        scan.seg = p.seg; scan.seg_len = p.seg_chunks * kC;
        e = launch_scan(scan, s);
        if (e != cudaSuccess) return e;
    }
    return launch<true>(my, p, s);
}

}  // namespace linear
}  // namespace gdn
