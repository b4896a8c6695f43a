// Gradients of linear attention on tensor cores, chunk by chunk (BackwardPass,
// linear_tc.cuh), from S entering and G = dL/d(state) leaving every chunk:
//     dq_i = scale ( lam^{i+1} S^T do_i + sum_{j<=i} lam^{i-j} (do_i.v_j) k_j )
//     dv_j = lam^{L-1-j} G k_j   + scale sum_{i>=j} lam^{i-j} (q_i.k_j) do_i
//     dk_j = lam^{L-1-j} G^T v_j + scale sum_{i>=j} lam^{i-j} (do_i.v_j) q_i
// (G carries the scale).  dq and dk sum over the v-heads of a group, in fp32
// tensor-core accumulators that live through the group's heads.
//
// Every (chunk, q/k head) is an item; a persistent CTA per SM takes items in
// turn.  A producer warp loads tiles, an MMA warp multiplies, 8 epilogue warps
// turn products into the next operands.  Tensor memory: the accumulators of dq
// and dk, one working accumulator R, and two bf16 operands A0, A1.  Per head:
//     R = dO V^T       -> A0 = masked, decayed;  A1 = scale lam^{i+1} dO
//     dq += A0 K + A1 S;           R = K Q^T   -> A0 masked, A1 = lam^{L-1-j} K
//     R = A0 dO + A1 G^T           -> dv out;     A1 = lam^{L-1-j} V
//     R = V dO^T                   -> A0 masked
//     dk += A0 Q + A1 G
// Each masked score, scaled row and state is rounded to bf16 (2^-8 of a term).
// Shared memory holds one head's tiles (V twice, so that the next head's can
// come while this one's is in use): 7 x 32 KB.
// Bound: HBM, 160 KB per chunk and v-head (V, dO, S, G, dv) and q, k, dq, dk per
// group, against nine 128^3 products (38 MFLOP).
#include "linear_tc.cuh"

namespace gdn {
namespace linear {
namespace {

constexpr int kEpiWarps = 8, kEpiThreads = 32 * kEpiWarps;
constexpr int kThreads = kEpiThreads + 64;
enum Buf { B_V0 = 0, B_V1, B_DO, B_K, B_S, B_Q, B_G, kBufs };
constexpr uint32_t OFF_MISC = kBufs * kTile;

struct Item {
    int64_t t0;
    int32_t L, j;
};

struct Misc {
    float up[8][32];  // per epilogue warp: lam^0 .. lam^31 of its head
    uint64_t full[kBufs], empty[kBufs];
    uint64_t item_full[2], item_empty[2];
    uint64_t mma_done, epi_done, clean, drain;
    Item item[2];
    uint32_t tmem;
    volatile int32_t abort;
};
constexpr uint32_t kSmem = OFF_MISC + sizeof(Misc) + 1024;
static_assert(kSmem <= 232448, "shared memory of an SM");

constexpr uint32_t TM_DQ = 0, TM_DK = 128, TM_R = 256, TM_A0 = 384, TM_A1 = 448;

struct Maps {
    CUtensorMap q, k, v, g;  // g: dO
};

// Tiles in the order of their first use.  n, u: items and v-heads so far.
__device__ void produce(const Maps &m, const BackwardPass &p, int64_t items, uint8_t *sm, Misc *ms, int G) {
    volatile int32_t *abort = &ms->abort;
    uint32_t cnt[kBufs] = {0, 0, 0, 0, 0, 0, 0};  // loads issued into each buffer
    bool ok = true;
    auto acquire = [&](int b) {
        if (ok && cnt[b] > 0) ok = role_wait(&ms->empty[b], (cnt[b] - 1) & 1, abort, p.err);
        if (ok) {
            ++cnt[b];
            mbar_arrive_expect_tx(&ms->full[b], kTile);
        }
        return ok;
    };
    uint32_t n = 0, u = 0;
    for (int64_t it = blockIdx.x; ok && it < items; it += gridDim.x) {
        const int64_t slot = it / p.Hqk;
        const int j = (int)(it - slot * p.Hqk);
        Span sp;
        if (!find_span(p.cu, p.N, p.T, kC, slot, p.err, sp) || sp.t1 <= sp.t0) continue;
        if (n >= 2 && !(ok = role_wait(&ms->item_empty[n & 1], ((n >> 1) - 1) & 1, abort, p.err))) break;
        ms->item[n & 1] = {sp.t0, (int32_t)(sp.t1 - sp.t0), j};
        mbar_arrive(&ms->item_full[n & 1]);
        ++n;
        for (int g = 0; g < G && ok; ++g, ++u) {
            const int h = j * G + g, bv = u & 1 ? B_V1 : B_V0;
            const int64_t img = (slot * p.Hv + h) * (int64_t)kTile;
            if (!acquire(bv)) break;
            load_tile(sm + bv * kTile, &m.v, &ms->full[bv], h, sp.t0);
            if (!acquire(B_DO)) break;
            load_tile(sm + B_DO * kTile, &m.g, &ms->full[B_DO], h, sp.t0);
            if (g == 0) {
                if (!acquire(B_K)) break;
                load_tile(sm + B_K * kTile, &m.k, &ms->full[B_K], j, sp.t0);
            }
            if (!acquire(B_S)) break;
            bulk_load(sm + B_S * kTile, p.dump_s + img, kTile, &ms->full[B_S]);
            if (g == 0) {
                if (!acquire(B_Q)) break;
                load_tile(sm + B_Q * kTile, &m.q, &ms->full[B_Q], j, sp.t0);
            }
            if (!acquire(B_G)) break;
            bulk_load(sm + B_G * kTile, p.dump_g + img, kTile, &ms->full[B_G]);
        }
    }
    if (ok && n >= 2) ok = role_wait(&ms->item_empty[n & 1], ((n >> 1) - 1) & 1, abort, p.err);
    if (ok) {
        ms->item[n & 1].L = -1;
        mbar_arrive(&ms->item_full[n & 1]);
        return;
    }
    // given up: let the loads in flight land before the CTA ends
    for (int b = 0; b < kBufs; ++b)
        if (cnt[b] > 0) mbar_wait_bounded(&ms->full[b], (cnt[b] - 1) & 1, kWaitLimit);
}

// Issues every MMA (one thread); steps: four per v-head, each ended by a commit
// to mma_done and followed by the epilogue's epi_done.
__device__ void multiply(const BackwardPass &p, uint32_t sbase, Misc *ms, uint32_t tmem, int G) {
    volatile int32_t *abort = &ms->abort;
    auto wait = [&](uint64_t &bar, uint32_t parity) { return role_wait(&bar, parity & 1, abort, p.err); };
    auto tile = [&](int b) { return sbase + b * kTile; };
    const uint32_t dq = tmem + TM_DQ, dk = tmem + TM_DK, R = tmem + TM_R, A0 = tmem + TM_A0, A1 = tmem + TM_A1;
    uint32_t u = 0, step = 0, dirty = 0;  // v-heads, epilogue steps, partial-chunk heads so far
    auto epi = [&]() {  // the epilogue's current step is done
        const bool ok = wait(ms->epi_done, step);
        ++step;
        tc_fence_after_sync();
        return ok;
    };
    for (uint32_t n = 0;; ++n) {
        if (!wait(ms->item_full[n & 1], n >> 1)) break;
        const int L = ms->item[n & 1].L;
        if (L < 0) {
            if (n > 0) mma_commit(&ms->mma_done);  // the last item's dq and dk
            return;
        }
        mbar_arrive(&ms->item_empty[n & 1]);
        bool ok = true;
        for (int g = 0; g < G; ++g, ++u) {
            const int bv = u & 1 ? B_V1 : B_V0;
            const bool first = g == 0, last = g == G - 1;
            ok = wait(ms->full[bv], u >> 1) && wait(ms->full[B_DO], u);
            if (ok && L < kC) ok = wait(ms->clean, dirty++);
            if (!ok) break;
            mma_kk(R, tile(B_DO), tile(bv), false);
            mma_commit(&ms->mma_done);
            ok = epi() && wait(ms->full[B_K], n) && wait(ms->full[B_S], u) && wait(ms->full[B_Q], n);
            if (!ok) break;
            mma_tm(dq, A0, tile(B_K), !first);
            mma_tm(dq, A1, tile(B_S), true);
            mma_commit(&ms->empty[B_S]);
            mma_kk(R, tile(B_K), tile(B_Q), false);
            mma_commit(&ms->mma_done);
            ok = epi() && wait(ms->full[B_G], u);
            if (!ok) break;
            if (last) mbar_arrive(&ms->empty[B_K]);  // read by these MMAs and this epilogue step
            mma_tm(R, A0, tile(B_DO), false);
            mma_tk(R, A1, tile(B_G), true);
            mma_commit(&ms->mma_done);
            if (!(ok = epi())) break;
            mma_kk(R, tile(bv), tile(B_DO), false);
            mma_commit(&ms->empty[B_DO]);
            mma_commit(&ms->empty[bv]);
            mma_commit(&ms->mma_done);
            if (!(ok = epi())) break;
            mma_tm(dk, A0, tile(B_Q), !first);
            mma_tm(dk, A1, tile(B_G), true);
            mma_commit(&ms->empty[B_G]);
            if (last) mma_commit(&ms->empty[B_Q]);
        }
        if (!ok) break;
    }
    // given up: let the MMAs in flight finish before tensor memory is freed
    mma_commit(&ms->drain);
    mbar_wait_bounded(&ms->drain, 0, kWaitLimit);
}

__device__ void epilogue(const BackwardPass &p, uint8_t *sm, Misc *ms, uint32_t tmem, int G) {
    volatile int32_t *abort = &ms->abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, half = warp >> 2;
    const int row = quad * 32 + lane;  // token of the chunk; columns 64 half ..
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
    float *up = ms->up[warp];
    auto wait = [&](uint64_t &bar, uint32_t parity) { return role_wait(&bar, parity & 1, abort, p.err); };
    uint32_t steps = 0;  // MMA steps waited for
    auto mma = [&]() {
        const bool ok = wait(ms->mma_done, steps);
        ++steps;
        tc_fence_after_sync();
        return ok;
    };
    auto done = [&]() {
        tmem_wait_st();
        tc_fence_before_sync();
        warp_arrive(&ms->epi_done);
    };
    // A0 = R times scale lam^|row - column| where the column is not after
    // (kLower) or not before the row, 0 elsewhere
    auto mask = [&](bool lower, float l2) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int cb = 2 * half + b;  // columns 32 cb ..
            uint32_t out[16];
            if (lower ? cb > quad : cb < quad) {
#pragma unroll
                for (int x = 0; x < 16; ++x) out[x] = 0u;
            } else {
                float v[32];
                tmem_ld32(trow + TM_R + 32 * cb, v);
                tmem_wait_ld();
                if (cb != quad) {
                    const float f = p.scale * exp2f(l2 * (float)(lower ? row - 32 * cb - 31 : 32 * cb - row));
#pragma unroll
                    for (int x = 0; x < 32; x += 4) {  // lower: lam^{31-x}, read backwards
                        const float4 w = *reinterpret_cast<const float4 *>(up + (lower ? 28 - x : x));
                        v[x] *= f * (lower ? w.w : w.x);
                        v[x + 1] *= f * (lower ? w.z : w.y);
                        v[x + 2] *= f * (lower ? w.y : w.z);
                        v[x + 3] *= f * (lower ? w.x : w.w);
                    }
                } else if (lower) {
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        v[x] = x <= lane ? v[x] * (p.scale * up[(lane - x) & 31]) : 0.f;
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        v[x] = x >= lane ? v[x] * (p.scale * up[(x - lane) & 31]) : 0.f;
                }
#pragma unroll
                for (int x = 0; x < 16; ++x) out[x] = pack_bf16(v[2 * x], v[2 * x + 1]);
            }
            tmem_st16u(trow + TM_A0 + 16 * cb, out);
        }
    };
    // A1 = this thread's half row of a tile, times f
    auto scaled = [&](int buf, float f) {
        const uint8_t *t = sm + buf * kTile + half * kSub;
        uint32_t out[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint4 v = *reinterpret_cast<const uint4 *>(t + sw128(row, 16 * c));
            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&in[q]));
                out[4 * c + q] = pack_bf16(a.x * f, a.y * f);
            }
        }
        tmem_st32u(trow + TM_A1 + 32 * half, out);
    };
    // this thread's half row of an accumulator to its token's row of dst
    auto write = [&](uint32_t col, void *dst, int64_t t0, int L, int H, int h, bool release) {
        float v[64];
        tmem_ld32(trow + col + 64 * half, *reinterpret_cast<float(*)[32]>(v));
        tmem_ld32(trow + col + 64 * half + 32, *reinterpret_cast<float(*)[32]>(v + 32));
        tmem_wait_ld();
        if (release) done();
        if (row >= L) return;
        __nv_bfloat16 *d = static_cast<__nv_bfloat16 *>(dst) + ((t0 + row) * H + h) * (int64_t)kD + 64 * half;
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) w[x] = pack_bf16(v[c + 2 * x], v[c + 2 * x + 1]);
            store_b256(d + c, w);
        }
    };
    // rows past a partial chunk's end: 0 times a neighbour's NaN would reach every sum over tokens
    auto clear = [&](int buf, int L) {
        uint8_t *t = sm + buf * kTile;
        for (int x = L * 8 + tid; x < kC * 8; x += kEpiThreads) {
            *reinterpret_cast<uint4 *>(t + x * 16) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(t + kSub + x * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
    };

    uint32_t u = 0;
    Item prev{0, -1, 0};
    for (uint32_t n = 0;; ++n) {
        if (!wait(ms->item_full[n & 1], n >> 1)) return;
        const Item im = ms->item[n & 1];
        if (im.L < 0) break;
        warp_arrive(&ms->item_empty[n & 1]);
        for (int g = 0; g < G; ++g, ++u) {
            const int h = im.j * G + g, bv = u & 1 ? B_V1 : B_V0;
            const float l2 = p.log_decay[h] * kLog2e;
            if (im.L < kC) {
                if (!wait(ms->full[bv], u >> 1) || !wait(ms->full[B_DO], u)) return;
                if (g == 0 && (!wait(ms->full[B_K], n) || !wait(ms->full[B_Q], n))) return;
                clear(bv, im.L);
                clear(B_DO, im.L);
                if (g == 0) {
                    clear(B_K, im.L);
                    clear(B_Q, im.L);
                }
                fence_proxy_async_smem();
                warp_arrive(&ms->clean);
            }
            __syncwarp();
            up[lane] = exp2f(l2 * (float)lane);
            __syncwarp();
            const float fi = p.scale * exp2f(l2 * (float)(row + 1));
            const float fj = row < im.L ? exp2f(l2 * (float)(im.L - 1 - row)) : 0.f;

            if (!mma()) return;  // R = dO V^T, and all of the previous item
            if (g == 0 && prev.L >= 0) {
                write(TM_DQ, p.dq, prev.t0, prev.L, p.Hqk, prev.j, false);
                write(TM_DK, p.dk, prev.t0, prev.L, p.Hqk, prev.j, false);
            }
            mask(true, l2);
            if (!wait(ms->full[B_DO], u)) return;
            scaled(B_DO, fi);
            done();
            if (!mma()) return;  // R = K Q^T
            mask(false, l2);
            if (!wait(ms->full[B_K], n)) return;
            scaled(B_K, fj);
            done();
            if (!mma()) return;  // R = dv
            if (!wait(ms->full[bv], u >> 1)) return;
            scaled(bv, fj);
            write(TM_R, p.dv, im.t0, im.L, p.Hv, h, true);
            if (!mma()) return;  // R = V dO^T
            mask(false, l2);
            done();
        }
        prev = im;
    }
    if (prev.L >= 0) {
        if (!mma()) return;
        write(TM_DQ, p.dq, prev.t0, prev.L, p.Hqk, prev.j, false);
        write(TM_DK, p.dk, prev.t0, prev.L, p.Hqk, prev.j, false);
    }
}

__global__ void __launch_bounds__(kThreads, 1)
    gdn_linear_backward_kernel(const __grid_constant__ Maps maps, BackwardPass p, int64_t items) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc *ms = reinterpret_cast<Misc *>(sm + OFF_MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.Hv / p.Hqk;
    if (tid == 0) {
        for (int b = 0; b < kBufs; ++b) {
            mbar_init(&ms->full[b], 1);
            mbar_init(&ms->empty[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ms->item_full[b], 1);
            mbar_init(&ms->item_empty[b], 1 + kEpiWarps);
        }
        mbar_init(&ms->mma_done, 1);
        mbar_init(&ms->epi_done, kEpiWarps);
        mbar_init(&ms->clean, kEpiWarps);
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
    if (warp == kEpiThreads / 32) {
        if (lane == 0) produce(maps, p, items, sm, ms, G);
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

cudaError_t launch_backward(const BackwardPass &p, cudaStream_t s) {
    Maps m;
    if (!make_tile_map_bf16_128(&m.q, p.q, p.T, p.Hqk, kC) || !make_tile_map_bf16_128(&m.k, p.k, p.T, p.Hqk, kC) ||
        !make_tile_map_bf16_128(&m.v, p.v, p.T, p.Hv, kC) || !make_tile_map_bf16_128(&m.g, p.dO, p.T, p.Hv, kC))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(gdn_linear_backward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmem);
    if (e != cudaSuccess) return e;
    const int64_t items = slots_of(p.T, p.N, kC) * p.Hqk, sms = device_sms();
    gdn_linear_backward_kernel<<<(unsigned)(items < sms ? items : sms), kThreads, kSmem, s>>>(m, p, items);
    return cudaGetLastError();
}

}  // namespace linear
}  // namespace gdn
