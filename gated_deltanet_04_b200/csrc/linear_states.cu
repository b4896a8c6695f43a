// Chunk states of linear attention on tensor cores (StatePass, linear_tc.cuh).
//
// One CTA walks the chunks of one (segment, head).  The fp32 state stays in
// tensor memory; each chunk's sum of outer products is one fresh tensor-core
// accumulator added to it by fp32 FMAs (the tensor core's own accumulation over
// thousands of chunks would truncate, and with a slow decay the loss would add
// up; for the same reason a slow decay acts by expm1, see Decay).
//
// Precision: y enters as it is (bf16); x times its decay weight is split into
// bf16 parts, hi + mid + lo, which together keep fp32's 24 bits: three MMA
// passes, wherever the sum goes into an fp32 state.  Where only bf16 images
// come of it (a segment that does not end its sequence), hi + mid do.
//
// The parts of x^T (128 rows, 64 tokens a stage) are the MMAs' first operand in
// tensor memory, one row per lane: the converting threads read x from shared
// memory with a lane per column, which transposes it on the way.
//
// Roles, on stages of 64 tokens: a producer warp loads x and y by TMA into a ring
// of five; two groups of 8 warps take stages in turn, each writing x's parts into a
// buffer of its own; an MMA warp sums a chunk's stages into an accumulator; 8
// warps add it to the state and store the image of the state that enters the
// next chunk.  (Tried: one set of warps doing all of it in turn, 3.3 us a chunk;
// x's parts in shared memory, whose bandwidth the products then need whole, 2.6;
// x from global memory to registers, a load's latency of 2,000 clocks a stage, 2.3.)
// Bound: HBM (64 KB in, 32 KB image out per chunk and head, y shared by the
// heads of a group through L2) against two or three products of 4.2 MFLOP.
// Measured, 65,536 tokens of 48 heads in 144 segments: images 356 us, 5.2 TB/s of
// 76 KB a chunk and head; sums 384 us, 2.2 us a chunk, where the conversion into three
// parts, the products and the ring take turns at the limit (without the conversion's
// arithmetic 18% less, without a third of the products 10%).
#include "linear_tc.cuh"

namespace gdn {
namespace linear {
namespace {

constexpr int kRows = 64;                    // tokens per stage
constexpr uint32_t kHalf = kRows * 128;      // 64 rows x 64 columns
constexpr uint32_t kPart = 2 * kHalf;        // 64 x 128 bf16
constexpr int kRing = 5;                     // stages of x and y
constexpr int kStateWarps = 8, kConvWarps = 16, kGroup = 8;  // warps; warps per converting group
constexpr int kStateThreads = kStateWarps * 32, kConvThreads = kConvWarps * 32;
constexpr int kThreads = kStateThreads + kConvThreads + 64;
constexpr uint32_t kStage = 2 * kPart;       // x, y
constexpr uint32_t kStateRow = 4 * kD + 16;  // a row of the fp32 state, staged in the ring
static_assert(kD * kStateRow <= kRing * kStage, "the state in the ring");
constexpr uint32_t OFF_IMAGE = kRing * kStage;
constexpr uint32_t OFF_MISC = OFF_IMAGE + kTile;

// Tensor memory columns: the state, two sums, and a buffer of two parts (32 columns
// each) per converting group.  A third part takes the first one's place once that has
// been multiplied.
constexpr uint32_t TM_S = 0, TM_SUM = 128, TM_PARTS = TM_SUM + 256;
constexpr int kSums = 2;

struct Misc {
    // of token pairs, a whole chunk's and the partial chunk's: as two bf16 parts, and in fp32
    alignas(16) uint32_t weight[2][2][kC / 2];
    alignas(16) float2 weight32[2][kC / 2];
    uint64_t raw_full[kRing], raw_empty[kRing], part_full[2], part_empty[2], third_full[2], first_empty[2],
        sum_full[2], sum_empty[2], drain;
    uint32_t tmem;
    volatile int32_t abort;
};
constexpr uint32_t kSmem = OFF_MISC + sizeof(Misc) + 1024;
static_assert(kSmem <= 232448, "shared memory of an SM");

// A launch's passes (blockIdx.y); all have the same N, T, H, cu and segments.
struct Passes {
    CUtensorMap x[2], y[2];
    StatePass p[2];
};

// The chunks of a segment in the pass's order: tokens t0 .. t0 + len - 1.
struct Walk {
    int64_t t0;
    int32_t len, nch;
    bool reverse;
    __device__ __forceinline__ int chunk(int it) const { return reverse ? nch - 1 - it : it; }
    __device__ __forceinline__ int length(int it) const { return min(len - chunk(it) * kC, kC); }
};

__device__ void produce(const CUtensorMap &tm_x, const CUtensorMap &tm_y, const Walk &w, int h, int hy, uint8_t *sm,
                        Misc *ms, int32_t *err) {
    uint32_t r = 0;  // stages so far
    for (int it = 0; it < w.nch; ++it) {
        const int L = w.length(it);
        for (int j0 = 0; j0 < L; j0 += kRows, ++r) {
            const int b = r % kRing;
            if (r >= kRing && !thread_wait(&ms->raw_empty[b], (r / kRing - 1) & 1, &ms->abort, err)) {
                // given up: let the loads in flight land before the CTA ends
                for (uint32_t x = r - kRing; x < r; ++x)
                    mbar_wait_bounded(&ms->raw_full[x % kRing], (x / kRing) & 1, kWaitLimit);
                return;
            }
            uint8_t *x = sm + b * kStage, *y = x + kPart;
            const int32_t t = (int32_t)w.t0 + w.chunk(it) * kC + j0;
            mbar_arrive_expect_tx(&ms->raw_full[b], kStage);
            tma_load_3d(x, &tm_x, &ms->raw_full[b], 0, h, t);
            tma_load_3d(x + kHalf, &tm_x, &ms->raw_full[b], 64, h, t);
            tma_load_3d(y, &tm_y, &ms->raw_full[b], 0, hy, t);
            tma_load_3d(y + kHalf, &tm_y, &ms->raw_full[b], 64, hy, t);
        }
    }
}

// Packed bf16 pairs: fused multiply-add, product, one rounding each.
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    return fma2(a, b, 0x80008000u);  // - 0: keeps the sign of a zero product
}

// The weights of a chunk of L tokens (0 past its end), of pairs of tokens; thread i <
// 64 has pair i.
__device__ __forceinline__ void make_weights(Misc *ms, int which, int i, int L, bool reverse, float l2,
                                             float x_scale) {
    auto weight = [&](int j) {
        if (j >= L) return 0.f;
        return reverse ? x_scale * exp2f(l2 * (float)(j + 1)) : exp2f(l2 * (float)(L - 1 - j));
    };
    const float2 f = make_float2(weight(2 * i), weight(2 * i + 1));
    ms->weight32[which][i] = f;
    const uint32_t hi = pack_bf16(f);
    const float2 g = unpack_bf16(hi);
    ms->weight[which][0][i] = hi;
    ms->weight[which][1][i] = pack_bf16(f.x - g.x, f.y - g.y);
}

__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Every second stage (group 0 or 1): x^T w into tensor memory, a thread per row
// (column of x) and 32 of the tokens.  Two parts, in packed bf16 arithmetic (fused
// multiply-adds, one rounding each): hi = x wh rounded; x wh - hi is exact (16 bits
// less the upper 8), so mid = x wm + (x wh - hi) is rounded once, 2^-17 of the
// product.  Three parts in fp32: each takes what the ones before left of x w, whose
// own rounding is fp32's.  A pair of lanes reads its two columns of two tokens, a
// token each, and swaps halves.
template <int kParts>
__device__ void convert(const Walk &w, uint8_t *sm, Misc *ms, uint32_t tlane, int group, int half, int tid,
                        int32_t *err) {
    struct At {  // stage s of chunk it
        int it, s;
    };
    auto advance = [&](At a) -> At {  // two stages on
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (a.it >= w.nch) break;
            if (a.s == 0 && w.length(a.it) > kRows) a.s = 1;
            else a = {a.it + 1, 0};
        }
        return a;
    };
    const int odd = tid & 1;
    const uint32_t swap = odd ? 0x3276u : 0x5410u;
    // tokens 32 half + 2 q + odd of a stage, this lane pair's columns: the swizzle repeats every 4 q
    const int row = tid & 127, col = row & ~1;
    uint32_t at_q[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) at_q[q] = (col >> 6) * kHalf + sw128(32 * half + 2 * q + odd, (col & 63) * 2);
    const uint32_t dst = tlane + TM_PARTS + 64 * group + 16 * half;
    At a{0, 0};
    if (group == 1) a = w.length(0) > kRows ? At{0, 1} : At{1, 0};
    for (uint32_t r = group; a.it < w.nch; r += 2) {
        const int L = w.length(a.it), left = L - a.s * kRows, b = r % kRing;
        const uint32_t(*wt)[kC / 2] = ms->weight[L < kC];
        const float2 *w32 = ms->weight32[L < kC];
        const int at = a.s * (kRows / 2) + 16 * half;
        if (!warp_wait(&ms->raw_full[b], (r / kRing) & 1, &ms->abort, err)) return;
        const uint8_t *x = sm + b * kStage;
        uint32_t in[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) in[q] = *reinterpret_cast<const uint32_t *>(x + at_q[q & 3] + (q >> 2) * 1024);
        if (left < kRows) {  // a neighbour's rows
#pragma unroll
            for (int q = 0; q < 16; ++q)
                if (32 * half + 2 * q + odd >= left) in[q] = 0u;
        }
#pragma unroll
        for (int q = 0; q < 16; ++q)  // this lane's column, two tokens
            in[q] = __byte_perm(in[q], __shfl_xor_sync(0xffffffffu, in[q], 1), swap);
        uint32_t lo[16];
#pragma unroll
        for (int q0 = 0; q0 < 16; q0 += 8) {
            uint32_t hi[8], mid[8];
            if constexpr (kParts == 2) {
#pragma unroll
                for (int q = 0; q < 8; q += 4) {
                    const uint4 h4 = *reinterpret_cast<const uint4 *>(&wt[0][at + q0 + q]);
                    const uint4 m4 = *reinterpret_cast<const uint4 *>(&wt[1][at + q0 + q]);
                    const uint32_t wh[4] = {h4.x, h4.y, h4.z, h4.w}, wm[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t v = in[q0 + q + e];
                        hi[q + e] = mul2(v, wh[e]);
                        mid[q + e] = fma2(v, wm[e], fma2(v, wh[e], hi[q + e] ^ 0x80008000u));
                    }
                }
            } else {
                const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
                for (int q = 0; q < 8; q += 2) {
                    const float4 f4 = *reinterpret_cast<const float4 *>(&w32[at + q0 + q]);
                    const float2 f[2] = {make_float2(f4.x, f4.y), make_float2(f4.z, f4.w)};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float2 left2 = fmul2(unpack_bf16(in[q0 + q + e]), f[e]);
                        hi[q + e] = pack_bf16(left2);
                        left2 = ffma2(unpack_bf16(hi[q + e]), minus, left2);
                        mid[q + e] = pack_bf16(left2);
                        lo[q0 + q + e] = pack_bf16(ffma2(unpack_bf16(mid[q + e]), minus, left2));
                    }
                }
            }
            // as late as can be: the MMAs of the other group's stage cover what follows
            if (q0 == 0 && r >= 2 && !warp_wait(&ms->part_empty[group], ((r >> 1) - 1) & 1, &ms->abort, err)) return;
            tc_fence_after_sync();
            tmem_st8u(dst + q0, hi);
            tmem_st8u(dst + 32 + q0, mid);
        }
        if (left < kRows) {  // y of the next sequence: 0 times its NaN would reach this sum
            uint8_t *y = sm + b * kStage + kPart;
            for (int k = tid; k < (kRows - left) * 16; k += 32 * kGroup)
                *reinterpret_cast<uint4 *>(y + (k & 1) * kHalf + left * 128 + (k >> 1) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before_sync();
        warp_arrive(&ms->part_full[group]);
        if (kParts == 3) {
            if (!warp_wait(&ms->first_empty[group], (r >> 1) & 1, &ms->abort, err)) return;
            tc_fence_after_sync();
            tmem_st16u(dst, lo);
            tmem_wait_st();
            tc_fence_before_sync();
            warp_arrive(&ms->third_full[group]);
        }
        a = advance(a);
    }
}

// Sums a chunk's stages: D = (hi + mid + lo)^T y, y MN-major.
template <int kParts>
__device__ void multiply(const Walk &w, uint32_t sbase, uint32_t tmem, Misc *ms, int32_t *err) {
    uint32_t r = 0, b = 0, lap = 0;  // stages so far; the ring's stage and lap
    const uint64_t y0 = desc_m(sbase + kPart, kHalf);
    bool ok = true;
    for (int it = 0; ok && it < w.nch; ++it) {
        const int L = w.length(it);
        const int sum = it % kSums;
        const uint32_t d = tmem + TM_SUM + 128 * sum;
        if (it >= kSums && !(ok = thread_wait(&ms->sum_empty[sum], (it / kSums - 1) & 1, &ms->abort, err))) break;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (s * kRows >= L) break;
            const uint32_t buf = r & 1;
            if (!(ok = thread_wait(&ms->raw_full[b], lap & 1, &ms->abort, err) &&
                       thread_wait(&ms->part_full[buf], (r >> 1) & 1, &ms->abort, err)))
                break;
            tc_fence_after_sync();
            const uint64_t y = y0 + b * (kStage >> 4);
            const uint32_t x = tmem + TM_PARTS + 64 * buf;
            auto part = [&](uint32_t a, bool first) {
#pragma unroll
                for (int ks = 0; ks < kRows / 16; ++ks)
                    mma_f16_ts(d, a + 8 * ks, step_m(y, ks), IDESC_KM, !first || ks);
            };
            part(x, s == 0);
            if (kParts == 3) mma_commit(&ms->first_empty[buf]);
            part(x + 32, false);
            if (kParts == 3) {
                if (!(ok = thread_wait(&ms->third_full[buf], (r >> 1) & 1, &ms->abort, err))) break;
                tc_fence_after_sync();
                part(x, false);
            }
            mma_commit(&ms->raw_empty[b]);
            mma_commit(&ms->part_empty[buf]);
            ++r;
            if (++b == kRing) {
                b = 0;
                ++lap;
            }
        }
        if (ok) mma_commit(&ms->sum_full[sum]);
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
    gdn_linear_states_kernel(const __grid_constant__ Passes passes) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc *ms = reinterpret_cast<Misc *>(sm + OFF_MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const StatePass &p = passes.p[blockIdx.y];
    const int h = blockIdx.x % p.H;
    const int64_t slot = blockIdx.x / p.H;
    const int64_t seg_len = p.seg ? p.seg_chunks * kC : (p.T > 0 ? p.T : 1);
    if (tid == kThreads - 1) check_range(p.cu, p.N, p.T, slot, p.err);
    Span sp;
    const bool some = find_span(p.cu, p.N, p.T, seg_len, slot, p.err, sp);
    const bool last = some && (p.reverse ? sp.s == 0 : sp.s == sp.count - 1);  // in the pass's order
    if (!some || (!kDump && last)) {  // nothing starts from a last segment's sum
        prior_done();
        return;
    }
    const int hy = h / (p.H / p.Hy);
    const int32_t len = (int32_t)(sp.t1 - sp.t0);
    const Walk w{sp.t0, len, (len + kC - 1) / kC, p.reverse};
    const float l2 = log2_decay(p.log_decay, h);
    const bool exact = !kDump || (last && p.mT);  // its sum goes into an fp32 state

    if (tid == 0) {
        for (int b = 0; b < kRing; ++b) {
            mbar_init(&ms->raw_full[b], 1);
            mbar_init(&ms->raw_empty[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ms->part_full[b], kGroup);
            mbar_init(&ms->part_empty[b], 1);
            mbar_init(&ms->third_full[b], kGroup);
            mbar_init(&ms->first_empty[b], 1);
            mbar_init(&ms->sum_full[b], 1);
            mbar_init(&ms->sum_empty[b], kStateWarps);
        }
        mbar_init(&ms->drain, 1);
        ms->abort = 0;
        fence_mbarrier_init();
    }
    if (tid < kC / 2) {
        make_weights(ms, 0, tid, kC, w.reverse, l2, p.x_scale);
        make_weights(ms, 1, tid, w.len % kC, w.reverse, l2, p.x_scale);
    }
    if (warp == 0) {
        tmem_alloc(&ms->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = ms->tmem;
    next_may_start();
    prior_done();

    if (warp >= kStateWarps) {
        const int cw = warp - kStateWarps;
        if (cw < kConvWarps) {
            // warp % 4 is the quarter of the lanes a warp may write
            const int quad = warp & 3, row = quad * 32 + lane, half = (cw >> 2) & 1, group = cw / kGroup;
            const uint32_t tlane = tmem + ((uint32_t)(quad * 32) << 16);
            if (w.nch > 0 && exact) convert<3>(w, sm, ms, tlane, group, half, row + 128 * half, p.err);
            else if (w.nch > 0) convert<2>(w, sm, ms, tlane, group, half, row + 128 * half, p.err);
        } else if (cw == kConvWarps) {
            if (lane == 0) produce(passes.x[blockIdx.y], passes.y[blockIdx.y], w, h, hy, sm, ms, p.err);
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
        if (kDump && p.seg && sp.count > 1) src = p.seg + (slot * p.H + h) * (int64_t)(kD * kD) + at;
        else if (kDump && p.m0 && st >= 0 && !state_fresh(p.map, sp.n))
            src = p.m0 + (st * p.H + h) * (int64_t)(kD * kD) + at;
#pragma unroll
        for (int c = 0; c < 64; c += 32) {  // a whole 128-byte line per thread at a time
            float v[32];
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
                uint32_t u[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                if (src) load_b256(src + c + x, u);
#pragma unroll
                for (int y = 0; y < 8; ++y) v[x + y] = __uint_as_float(u[y]);
            }
            tmem_st32(trow + TM_S + c, v);
            if (kDump && w.nch > 0) {
                draw(c, v);
                draw(c + 16, v + 16);
            }
        }
        tmem_wait_st();
        if (kDump && w.nch > 0) store_image(0);
        const float g = p.log_decay[h];
        const Decay full(g * (float)kC);  // a product of its own, once per chunk: see Decay
        bool ok = true;
        for (int it = 0; it < w.nch; ++it) {
            // every warp goes on after a wait given up, so that the barriers stay whole
            const int sum = it % kSums;
            if (ok) ok = warp_wait(&ms->sum_full[sum], (it / kSums) & 1, &ms->abort, p.err);
            tc_fence_after_sync();
            const bool more = kDump && it + 1 < w.nch;
            if (more) {
                if (tid == 0) bulk_wait_read_all();  // the image buffer is free again
                state_barrier();
            }
            const int L = w.length(it);
            const Decay dec = L < kC ? Decay(g * (float)L) : full;
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
                float v[16], d[16];
                tmem_ld16(trow + TM_S + c, v);
                tmem_ld16(trow + TM_SUM + 128 * sum + c, d);
                tmem_wait_ld();
                if (c == 48) {  // the sum has been read
                    tc_fence_before_sync();
                    warp_arrive(&ms->sum_empty[sum]);
                }
                auto add = [&](auto slow) {  // a uniform choice
#pragma unroll
                    for (int x = 0; x < 16; x += 2) {
                        const float2 s = dec.plus<decltype(slow)::value>(make_float2(v[x], v[x + 1]),
                                                                         make_float2(d[x], d[x + 1]));
                        v[x] = s.x;
                        v[x + 1] = s.y;
                    }
                };
                if (dec.slow) add(std::true_type{});
                else add(std::false_type{});
                tmem_st16(trow + TM_S + c, v);
                if (more) draw(c, v);
            }
            tmem_wait_st();
            if (more) store_image(it + 1);
        }
        float *dst = kDump ? (last && p.mT && st >= 0 ? p.mT + (st * p.H + h) * (int64_t)(kD * kD) : nullptr)
                           : p.seg + (slot * p.H + h) * (int64_t)(kD * kD);
        // through the ring, which is free now: its rows 16 bytes apart in the banks, each a
        // bulk copy (rows straight from registers are a line per thread: 4,200 clocks)
        if (dst) {
            float *stage = reinterpret_cast<float *>(sm + row * kStateRow) + 64 * half;
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                float v[32];
                tmem_ld32(trow + TM_S + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 32; x += 4)
                    *reinterpret_cast<float4 *>(stage + c + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
            }
            fence_proxy_async_smem();
            state_barrier();
            if (ok && tid < kD) {
                bulk_store(dst + tid * kD, sm + tid * kStateRow, kD * sizeof(float));
                bulk_commit();
            }
        }
        if (tid < kD) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <bool kDump>
cudaError_t launch(const Passes &passes, int count, bool after, cudaStream_t s) {
    const StatePass &p = passes.p[0];
    const int64_t len = p.seg ? p.seg_chunks * kC : (p.T > 0 ? p.T : 1);
    const int64_t blocks = slots_of(p.T, p.N, len) * p.H;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(gdn_linear_states_kernel<kDump>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    return launch_after(gdn_linear_states_kernel<kDump>, after, dim3((unsigned)blocks, count), kThreads, kSmem, s,
                        passes);
}

}  // namespace

int device_sms() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

// Segments, when one sequence could keep a CTA busy for much longer than an even
// share of all chunks would (the segment sums walk the chunks a second time): as
// long as the share, so that one wave of 148 CTAs has them all.  Measured with 48 heads and
// one sequence, sums + scan + images against one segment: 4,096 tokens 31 + 6 + 33 us
// and 81, 65,536 tokens 384 + 8 + 356 and 1,142.  Two passes at once, where the rule
// says one segment: 57 + 10 + 54 and 59, 851 + 11 + 715 and 1,138.
int64_t state_seg_chunks(int32_t N, int64_t T, int32_t H, int passes) {
    const int64_t longest = T / kC + 1, all = (T / kC + N) * H * passes, share = all / 148;
    if (N <= 0 || T <= 0 || longest <= 3 * share + 2) return 0;
    const int64_t len = (all + 147) / 148;
    return len < 4 ? 4 : len;
}

size_t state_seg_bytes(int32_t N, int64_t T, int32_t H, int passes) {
    const int64_t c = state_seg_chunks(N, T, H, passes);
    return c ? (size_t)slots_of(T, N, c * kC) * H * kD * kD * 4 : 0;
}

size_t state_dump_bytes(int32_t N, int64_t T, int32_t H) { return (size_t)slots_of(T, N, kC) * H * kTile; }

cudaError_t launch_states(const StatePass *p, int passes, cudaStream_t s) {
    Passes all{};
    for (int i = 0; i < passes; ++i) {
        const int64_t Tm = p[i].T > 0 ? p[i].T : 1;
        if (!make_tile_map_bf16_128(&all.x[i], p[i].x, Tm, p[i].H, kRows) ||
            !make_tile_map_bf16_128(&all.y[i], p[i].y, Tm, p[i].Hy, kRows))
            return cudaErrorInvalidValue;
        all.p[i] = p[i];
    }
    if (p[0].seg) {
        cudaError_t e = launch<false>(all, passes, false, s);
        if (e != cudaSuccess) return e;
        Pass scan[2];
        for (int i = 0; i < passes; ++i) {
            const StatePass &a = p[i];
            Pass &b = scan[i] = Pass{};
            b.H = a.H; b.Da = kD; b.Dc = kD; b.log_decay = a.log_decay; b.reverse = a.reverse;
            b.m0 = a.m0; b.map = a.map; b.cu = a.cu; b.N = a.N; b.T = a.T; b.err = a.err;
            b.seg = a.seg; b.seg_len = a.seg_chunks * kC;
        }
        e = launch_scan(scan, passes, s);
        if (e != cudaSuccess) return e;
    }
    return launch<true>(all, passes, p[0].seg != nullptr, s);
}

}  // namespace linear
}  // namespace gdn
