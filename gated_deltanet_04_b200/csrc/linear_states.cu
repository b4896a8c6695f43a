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
// Roles, on stages of 64 tokens: a producer warp loads x and y by TMA into a
// ring; two groups of 8 warps take stages in turn, turning x in place into hi
// and writing mid and lo beside it (one group alone was bound by the latency of
// its steps, 2.2 us a chunk with or without lo); an MMA warp sums a chunk's
// stages into one of two accumulators; 8 warps add it to the state and store
// the image of the state that enters the next chunk.
// Bound: HBM (64 KB in, 32 KB image out per chunk and head, y shared by the
// heads of a group through L2) against two or three products of 4.2 MFLOP.
#include "linear_tc.cuh"

namespace gdn {
namespace linear {
namespace {

constexpr int kRows = 64;                    // tokens per stage
constexpr uint32_t kHalf = kRows * 128;      // 64 rows x 64 columns
constexpr uint32_t kPart = 2 * kHalf;        // 64 x 128 bf16
constexpr int kRing = 4;
constexpr int kStateWarps = 8, kConvWarps = 8, kConvGroups = 2;
constexpr int kStateThreads = kStateWarps * 32, kConvThreads = kConvWarps * 32;
constexpr int kThreads = kStateThreads + kConvGroups * kConvThreads + 64;
constexpr uint32_t TM_S = 256;  // tensor memory: two sums, the state
constexpr uint32_t OFF_PARTS = kRing * 2 * kPart;       // [2][mid, lo]
constexpr uint32_t OFF_IMAGE = OFF_PARTS + 4 * kPart;
constexpr uint32_t OFF_MISC = OFF_IMAGE + kTile;

struct Misc {
    uint64_t raw_full[kRing], raw_empty[kRing], part_full[2], part_empty[2], sum_full[2], sum_empty[2], drain;
    uint32_t tmem;
    volatile int32_t abort;
};
constexpr uint32_t kSmem = OFF_MISC + sizeof(Misc) + 1024;
static_assert(kSmem <= 232448, "shared memory of an SM");

// The chunks of a segment in the pass's order.
struct Walk {
    int64_t t0, t1;
    int nch;
    bool reverse;
    __device__ __forceinline__ int chunk(int it) const { return reverse ? nch - 1 - it : it; }
    __device__ __forceinline__ int64_t start(int it) const { return t0 + (int64_t)chunk(it) * kC; }
    __device__ __forceinline__ int length(int it) const {
        const int64_t left = t1 - start(it);
        return left < kC ? (int)left : kC;
    }
};

__device__ void produce(const CUtensorMap &tm_x, const CUtensorMap &tm_y, const Walk &w, int h, int hy, uint8_t *sm,
                        Misc *ms, int32_t *err) {
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
            uint8_t *y = sm + b * 2 * kPart, *x = y + kPart;
            const int32_t t = (int32_t)(w.start(it) + j0);
            mbar_arrive_expect_tx(&ms->raw_full[b], 2 * kPart);
            tma_load_3d(x, &tm_x, &ms->raw_full[b], 0, h, t);
            tma_load_3d(x + kHalf, &tm_x, &ms->raw_full[b], 64, h, t);
            tma_load_3d(y, &tm_y, &ms->raw_full[b], 0, hy, t);
            tma_load_3d(y + kHalf, &tm_y, &ms->raw_full[b], 64, hy, t);
        }
    }
}

// x w = hi + mid + lo: hi in place, the others into the parts buffer of the
// group, which takes every second stage.
__device__ void convert(const Walk &w, float l2, float x_scale, int parts, uint8_t *sm, Misc *ms, int group, int tid,
                        int32_t *err) {
    const int r0 = tid >> 3, piece = (tid & 7) * 16;  // rows r0 and r0 + 32 of a stage
    const float2 minus = make_float2(-1.f, -1.f);
    uint32_t r = 0;  // stages so far, of both groups
    // weight of row j of a chunk of L tokens (0 past its end)
    auto weight = [&](int j, int L) {
        if (j >= L) return 0.f;
        return w.reverse ? x_scale * exp2f(l2 * (float)(j + 1)) : exp2f(l2 * (float)(L - 1 - j));
    };
    float wfull[4];  // of whole chunks
#pragma unroll
    for (int i = 0; i < 4; ++i) wfull[i] = weight(r0 + 32 * i, kC);
    for (int it = 0; it < w.nch; ++it) {
        const int L = w.length(it);
        for (int s = 0; s * kRows < L; ++s, ++r) {
            if ((r & 1) != group) continue;
            const int b = r % kRing;
            if (!role_wait(&ms->raw_full[b], (r / kRing) & 1, &ms->abort, err)) return;
            if (r >= 2 && !role_wait(&ms->part_empty[r & 1], ((r >> 1) - 1) & 1, &ms->abort, err)) return;
            uint8_t *y = sm + b * 2 * kPart, *x = y + kPart, *mid = sm + OFF_PARTS + (r & 1) * 2 * kPart;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = s * kRows + r0 + 32 * i;
                const float f = L == kC ? (s ? wfull[2 + i] : wfull[i]) : weight(j, L);
#pragma unroll
                for (int sub = 0; sub < 2; ++sub) {
                    const uint32_t at = sub * kHalf + (r0 + 32 * i) * 128 + piece;
                    uint32_t a[4] = {0u, 0u, 0u, 0u}, m[4] = {0u, 0u, 0u, 0u}, l[4] = {0u, 0u, 0u, 0u};
                    if (j < L) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(x + at);
                        const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float2 e = fmul2(unpack_bf16(in[q]), make_float2(f, f));
                            a[q] = pack_bf16(e);
                            const float2 d = ffma2(unpack_bf16(a[q]), minus, e);
                            m[q] = pack_bf16(d);
                            if (parts == 3) l[q] = pack_bf16(ffma2(unpack_bf16(m[q]), minus, d));
                        }
                    } else {  // rows of the next sequence: y too, or its NaN would reach this sum
                        *reinterpret_cast<uint4 *>(y + at) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    *reinterpret_cast<uint4 *>(x + at) = make_uint4(a[0], a[1], a[2], a[3]);
                    *reinterpret_cast<uint4 *>(mid + at) = make_uint4(m[0], m[1], m[2], m[3]);
                    if (parts == 3) *reinterpret_cast<uint4 *>(mid + kPart + at) = make_uint4(l[0], l[1], l[2], l[3]);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&ms->part_full[r & 1]);
        }
    }
}

// D (+)= x^T y over a stage's 64 tokens, both MN-major.
__device__ __forceinline__ void mma_stage(uint32_t d, uint32_t x, uint32_t y, bool acc) {
#pragma unroll
    for (int ks = 0; ks < kRows / 16; ++ks)
        mma_f16_ss(d, make_sdesc(x + ks * 2048, kHalf, 1024), make_sdesc(y + ks * 2048, kHalf, 1024), IDESC_MM,
                   acc || ks);
}

__device__ void multiply(const Walk &w, int parts, uint32_t sbase, uint32_t tmem, Misc *ms, int32_t *err) {
    uint32_t r = 0;
    bool ok = true;
    for (int it = 0; ok && it < w.nch; ++it) {
        const int L = w.length(it);
        const uint32_t d = tmem + 128 * (it & 1);
        if (it >= 2 && !(ok = role_wait(&ms->sum_empty[it & 1], ((it >> 1) - 1) & 1, &ms->abort, err))) break;
        for (int j0 = 0; j0 < L; j0 += kRows, ++r) {
            if (!(ok = role_wait(&ms->part_full[r & 1], (r >> 1) & 1, &ms->abort, err))) break;
            tc_fence_after_sync();
            const uint32_t y = sbase + (r % kRing) * 2 * kPart, mid = sbase + OFF_PARTS + (r & 1) * 2 * kPart;
            mma_stage(d, y + kPart, y, j0 > 0);
            mma_stage(d, mid, y, true);
            if (parts == 3) mma_stage(d, mid + kPart, y, true);
            mma_commit(&ms->raw_empty[r % kRing]);
            mma_commit(&ms->part_empty[r & 1]);
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
    gdn_linear_states_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y,
                             StatePass p) {
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
    const Walk w{sp.t0, sp.t1, (int)((sp.t1 - sp.t0 + kC - 1) / kC), p.reverse};
    const float l2 = p.log_decay[h] * kLog2e;
    const int parts = kDump && !(last && p.mT) ? 2 : 3;

    if (tid == 0) {
        for (int b = 0; b < kRing; ++b) {
            mbar_init(&ms->raw_full[b], 1);
            mbar_init(&ms->raw_empty[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ms->part_full[b], kConvThreads);
            mbar_init(&ms->part_empty[b], 1);
            mbar_init(&ms->sum_full[b], 1);
            mbar_init(&ms->sum_empty[b], kStateThreads);
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
        if (cw < kConvGroups * kConvWarps)
            convert(w, l2, p.x_scale, parts, sm, ms, cw / kConvWarps, (tid - kStateThreads) % kConvThreads, p.err);
        else if (cw == kConvGroups * kConvWarps) {
            if (lane == 0) produce(tm_x, tm_y, w, h, hy, sm, ms, p.err);
        } else if (lane == 0) {
            multiply(w, parts, smem_u32(sm), tmem, ms, p.err);
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
            mbar_arrive(&ms->sum_empty[it & 1]);
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
    if (!make_tile_map_bf16_128(&mx, p.x, Tm, p.H, kRows) || !make_tile_map_bf16_128(&my, p.y, Tm, p.Hy, kRows))
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
