// Outputs of linear attention on tensor cores, chunk by chunk (OutPass,
// linear_tc.cuh), from the states entering every chunk:
//     o_i = scale ( lam^{i+1} S q_i + sum_{j <= i} lam^{i-j} (q_i . k_j) v_j )
//
// Every (chunk, q/k head) is an item of its own; a persistent CTA per SM takes
// items in turn and, within one, the v-heads that share the q/k head, whose
// Q K^T is computed once.  Roles: a producer warp (TMA loads), an MMA warp, and
// 8 epilogue warps.  Per v-head the tensor core does Q S^T (accumulator Ox) and
// P V (Oi), P = Q K^T times the decay mask, bf16, in tensor memory; the epilogue
// adds Oi + scale lam^{i+1} Ox in fp32 and rounds once.  P and S are rounded to
// bf16 (half a step, 2^-8 of each term: as much as the output's own rounding).
//
// The epilogue makes the next head's P while the tensor core works on this
// one.  Shared memory: Q twice, K, and a ring of four tiles for V and S.
// Bound: HBM, 96 KB per chunk and v-head (V, S, o) and Q, K once per group: 118 KB
// with three v-heads a group.  Measured, 48 heads: 65,536 tokens 465 us, 6.2 TB/s;
// 4,096 tokens 39 us, where 512 items on 148 SMs leave the last of four turns half empty.
#include "linear_tc.cuh"

namespace gdn {
namespace linear {
namespace {

constexpr int kEpiWarps = 8, kEpiThreads = 32 * kEpiWarps;
constexpr int kThreads = kEpiThreads + 64;
constexpr int kRing = 4;
constexpr uint32_t OFF_Q = 0, OFF_K = 2 * kTile, OFF_RING = 3 * kTile, OFF_MISC = OFF_RING + kRing * kTile;

// What an item is; L < 0 ends the CTA's work.
struct Item {
    int64_t t0;
    int32_t L, j;
};

struct Misc {
    float pow[8][32];  // per epilogue warp: lam^31 .. lam^0 of its head
    uint64_t full_q[2], empty_q[2], full_k, empty_k, full_v[kRing], empty_v[kRing];
    uint64_t qk_done, qk_free, p_ready[2], o_done, o_free, drain;
    Item item[2];
    uint32_t tmem;
    volatile int32_t abort;
};
constexpr uint32_t kSmem = OFF_MISC + sizeof(Misc) + 1024;
static_assert(kSmem <= 232448, "shared memory of an SM");

// TMEM columns: Q K^T, two P (bf16 pairs), Oi, Ox.
constexpr uint32_t TM_QK = 0, TM_P = 128, TM_OI = 256, TM_OX = 384;

// Loads the tiles of this CTA's items in the order the MMA warp uses them.
__device__ void produce(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v, const OutPass &p,
                        int64_t items, uint8_t *sm, Misc *ms, int G) {
    uint32_t n = 0, r = 0;  // items and ring tiles so far
    volatile int32_t *abort = &ms->abort;
    auto wait_q = [&]() { return n < 2 || thread_wait(&ms->empty_q[n & 1], ((n >> 1) - 1) & 1, abort, p.err); };
    auto wait_ring = [&]() {
        return r < kRing || thread_wait(&ms->empty_v[r % kRing], (r / kRing - 1) & 1, abort, p.err);
    };
    bool ok = true, k_issued = true;
    for (int64_t it = blockIdx.x; ok && it < items; it += gridDim.x) {
        const int64_t slot = it / p.Hqk;
        const int j = (int)(it - slot * p.Hqk);
        Span sp;
        if (!find_span(p.cu, p.N, p.T, kC, slot, p.err, sp) || sp.t1 <= sp.t0) continue;
        if (!(ok = wait_q())) break;
        ms->item[n & 1] = {sp.t0, (int32_t)(sp.t1 - sp.t0), j};
        mbar_arrive_expect_tx(&ms->full_q[n & 1], kTile);
        load_tile(sm + OFF_Q + (n & 1) * kTile, &tm_q, &ms->full_q[n & 1], j, sp.t0);
        k_issued = ok = n < 1 || thread_wait(&ms->empty_k, (n - 1) & 1, abort, p.err);
        ++n;
        if (!ok) break;
        mbar_arrive_expect_tx(&ms->full_k, kTile);
        load_tile(sm + OFF_K, &tm_k, &ms->full_k, j, sp.t0);
        for (int g = 0; g < G; ++g) {
            const int h = j * G + g;
            if (!(ok = wait_ring())) break;
            mbar_arrive_expect_tx(&ms->full_v[r % kRing], kTile);
            load_tile(sm + OFF_RING + (r % kRing) * kTile, &tm_v, &ms->full_v[r % kRing], h, sp.t0);
            ++r;
            if (!(ok = wait_ring())) break;
            mbar_arrive_expect_tx(&ms->full_v[r % kRing], kTile);
            bulk_load(sm + OFF_RING + (r % kRing) * kTile, p.dump + (slot * p.Hv + h) * (int64_t)kTile, kTile,
                      &ms->full_v[r % kRing]);
            ++r;
        }
    }
    if (ok && (ok = wait_q())) {
        ms->item[n & 1].L = -1;
        mbar_arrive(&ms->full_q[n & 1]);
    }
    if (ok) return;
    // given up: let the loads in flight land before the CTA ends
    for (uint32_t x = n > 2 ? n - 2 : 0; x < n; ++x) mbar_wait_bounded(&ms->full_q[x & 1], (x >> 1) & 1, kWaitLimit);
    const uint32_t nk = k_issued ? n : n - 1;
    if (nk > 0) mbar_wait_bounded(&ms->full_k, (nk - 1) & 1, kWaitLimit);
    for (uint32_t x = r > kRing ? r - kRing : 0; x < r; ++x)
        mbar_wait_bounded(&ms->full_v[x % kRing], (x / kRing) & 1, kWaitLimit);
}

// Issues every MMA (one thread).
__device__ void multiply(const OutPass &p, uint32_t sbase, Misc *ms, uint32_t tmem, int G) {
    volatile int32_t *abort = &ms->abort;
    uint32_t u = 0, r = 0;  // v-heads and ring tiles so far
    auto wait = [&](uint64_t &bar, uint32_t parity) { return thread_wait(&bar, parity & 1, abort, p.err); };
    for (uint32_t n = 0;; ++n) {
        if (!wait(ms->full_q[n & 1], n >> 1)) break;
        if (ms->item[n & 1].L < 0) return;
        const uint32_t q = sbase + OFF_Q + (n & 1) * kTile;
        if (!wait(ms->full_k, n) || (n > 0 && !wait(ms->qk_free, n - 1))) break;
        tc_fence_after_sync();
        mma_kk(tmem + TM_QK, q, sbase + OFF_K, false);
        mma_commit(&ms->qk_done);
        mma_commit(&ms->empty_k);
        bool ok = true;
        for (int g = 0; g < G; ++g, ++u, r += 2) {
            const uint32_t rv = r % kRing, rs = (r + 1) % kRing;
            ok = wait(ms->full_v[rs], (r + 1) / kRing) && (u == 0 || wait(ms->o_free, u - 1));
            if (!ok) break;
            tc_fence_after_sync();
            mma_kk(tmem + TM_OX, q, sbase + OFF_RING + rs * kTile, false);
            mma_commit(&ms->empty_v[rs]);
            if (g == G - 1) mma_commit(&ms->empty_q[n & 1]);
            ok = wait(ms->full_v[rv], r / kRing) && wait(ms->p_ready[u & 1], u >> 1);
            if (!ok) break;
            tc_fence_after_sync();
            mma_tm(tmem + TM_OI, tmem + TM_P + 64 * (u & 1), sbase + OFF_RING + rv * kTile, false);
            mma_commit(&ms->empty_v[rv]);
            mma_commit(&ms->o_done);
        }
        if (!ok) break;
    }
    // given up: let the MMAs in flight finish before tensor memory is freed
    mma_commit(&ms->drain);
    mbar_wait_bounded(&ms->drain, 0, kWaitLimit);
}

__device__ void epilogue(const OutPass &p, uint8_t *sm, Misc *ms, uint32_t tmem, int G) {
    volatile int32_t *abort = &ms->abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, half = warp >> 2;
    const int i = quad * 32 + lane;  // token of the chunk; its columns 64 half ..
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
    float *pow = ms->pow[warp];
    auto wait = [&](uint64_t &bar, uint32_t parity) { return warp_wait(&bar, parity & 1, abort, p.err); };

    // P of v-head number u: Q K^T times scale lam^{i-j}, j <= i
    auto make_p = [&](uint32_t u, float l2) {
        __syncwarp();
        pow[lane] = exp2f(l2 * (float)(31 - lane));
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int jb = 2 * half + b;  // columns 32 jb ..
            uint32_t out[16];
            if (jb > quad) {
#pragma unroll
                for (int x = 0; x < 16; ++x) out[x] = 0u;
            } else {
                float v[32];
                tmem_ld32(trow + TM_QK + 32 * jb, v);
                tmem_wait_ld();
                if (jb < quad) {  // i - j = (i - 32 jb - 31) + (31 - x), both >= 0
                    const float f = p.scale * exp2f(l2 * (float)(i - 32 * jb - 31));
#pragma unroll
                    for (int x = 0; x < 32; x += 4) {
                        const float4 w = *reinterpret_cast<const float4 *>(pow + x);
                        v[x] *= f * w.x;
                        v[x + 1] *= f * w.y;
                        v[x + 2] *= f * w.z;
                        v[x + 3] *= f * w.w;
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        v[x] = x <= lane ? v[x] * (p.scale * pow[(31 - lane + x) & 31]) : 0.f;
                }
#pragma unroll
                for (int x = 0; x < 16; ++x) out[x] = pack_bf16(v[2 * x], v[2 * x + 1]);
            }
            tmem_st16u(trow + TM_P + 64 * (u & 1) + 16 * jb, out);
        }
        tmem_wait_st();
    };
    // o of v-head number u
    auto write_o = [&](uint32_t u, int64_t t0, int L, int h, float l2) -> bool {
        if (!wait(ms->o_done, u)) return false;
        tc_fence_after_sync();
        float a[64], b[64];
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
            tmem_ld32(trow + TM_OI + 64 * half + c, *reinterpret_cast<float(*)[32]>(a + c));
            tmem_ld32(trow + TM_OX + 64 * half + c, *reinterpret_cast<float(*)[32]>(b + c));
        }
        tmem_wait_ld();
        tc_fence_before_sync();
        warp_arrive(&ms->o_free);
        if (i >= L) return true;
        const float f = p.scale * exp2f(l2 * (float)(i + 1));
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.o) + ((t0 + i) * p.Hv + h) * (int64_t)kD + 64 * half;
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x)
                w[x] = pack_bf16(fmaf(f, b[c + 2 * x], a[c + 2 * x]), fmaf(f, b[c + 2 * x + 1], a[c + 2 * x + 1]));
            store_b256(dst + c, w);
        }
        return true;
    };

    uint32_t u = 0, r = 0;
    int64_t prev_t0 = 0;
    int prev_L = 0, prev_h = -1;
    float prev_l2 = 0.f;
    for (uint32_t n = 0;; ++n) {
        if (!wait(ms->full_q[n & 1], n >> 1)) return;
        const Item im = ms->item[n & 1];
        if (im.L < 0) break;
        warp_arrive(&ms->empty_q[n & 1]);
        if (!wait(ms->qk_done, n)) return;
        tc_fence_after_sync();
        for (int g = 0; g < G; ++g, ++u, r += 2) {
            const int h = im.j * G + g;
            const float l2 = log2_decay(p.log_decay, h);
            if (im.L < kC) {  // V rows of the next sequence: 0 times their NaN would reach every row
                if (!wait(ms->full_v[r % kRing], r / kRing)) return;
                uint8_t *v = sm + OFF_RING + (r % kRing) * kTile;
                for (int x = im.L * 8 + tid; x < kC * 8; x += kEpiThreads) {
                    *reinterpret_cast<uint4 *>(v + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4 *>(v + kSub + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            make_p(u, l2);
            tc_fence_before_sync();
            warp_arrive(&ms->p_ready[u & 1]);
            if (g == G - 1) warp_arrive(&ms->qk_free);
            if (prev_h >= 0 && !write_o(u - 1, prev_t0, prev_L, prev_h, prev_l2)) return;
            prev_t0 = im.t0;
            prev_L = im.L;
            prev_h = h;
            prev_l2 = l2;
        }
    }
    if (prev_h >= 0) write_o(u - 1, prev_t0, prev_L, prev_h, prev_l2);
}

__global__ void __launch_bounds__(kThreads, 1)
    gdn_linear_out_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, OutPass p, int64_t items) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc *ms = reinterpret_cast<Misc *>(sm + OFF_MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.Hv / p.Hqk;

    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ms->full_q[b], 1);
            mbar_init(&ms->empty_q[b], 1 + kEpiWarps);
            mbar_init(&ms->p_ready[b], kEpiWarps);
        }
        mbar_init(&ms->full_k, 1);
        mbar_init(&ms->empty_k, 1);
        for (int b = 0; b < kRing; ++b) {
            mbar_init(&ms->full_v[b], 1);
            mbar_init(&ms->empty_v[b], 1);
        }
        mbar_init(&ms->drain, 1);
        mbar_init(&ms->qk_done, 1);
        mbar_init(&ms->qk_free, kEpiWarps);
        mbar_init(&ms->o_done, 1);
        mbar_init(&ms->o_free, kEpiWarps);
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
    prior_done();
    if (warp == kEpiThreads / 32) {
        if (lane == 0) produce(tm_q, tm_k, tm_v, p, items, sm, ms, G);
    } else if (warp == kEpiThreads / 32 + 1) {
        if (lane == 0) multiply(p, smem_u32(sm), ms, tmem, G);
    } else {
        epilogue(p, sm, ms, tmem, G);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_out(const OutPass &p, cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    if (!make_tile_map_bf16_128(&mq, p.q, p.T, p.Hqk, kC) || !make_tile_map_bf16_128(&mk, p.k, p.T, p.Hqk, kC) ||
        !make_tile_map_bf16_128(&mv, p.v, p.T, p.Hv, kC))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(gdn_linear_out_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int64_t items = slots_of(p.T, p.N, kC) * p.Hqk, sms = device_sms();
    return launch_after(gdn_linear_out_kernel, true, dim3((unsigned)(items < sms ? items : sms)), kThreads, kSmem, s,
                        mq, mk, mv, p, items);
}

}  // namespace linear
}  // namespace gdn
