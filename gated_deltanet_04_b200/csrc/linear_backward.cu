// Gradients of linear attention on tensor cores, chunk by chunk (BackwardPass,
// linear_tc.cuh), from S entering and G = dL/d(state) leaving every chunk:
//     dq_i = scale ( lam^{i+1} S^T do_i + sum_{j<=i} lam^{i-j} (do_i.v_j) k_j )
//     dv_j = lam^{L-1-j} G k_j   + scale sum_{i>=j} lam^{i-j} (q_i.k_j) do_i
//     dk_j = lam^{L-1-j} G^T v_j + scale sum_{i>=j} lam^{i-j} (do_i.v_j) q_i
// (G carries the scale).  dq and dk sum over the v-heads of a group, in fp32
// tensor-core accumulators that live through the group's heads.
//
// Every (chunk, q/k head) is an item; a persistent CTA per SM takes items in
// turn.  A producer warp loads tiles, an MMA warp multiplies, 16 epilogue warps
// (a row's 32 columns per thread) work between the products.  Per v-head, with
// two working accumulators T0, T1 in tensor memory beside those of dq and dk:
//     T0 = K Q^T    -> P^T (decayed, masked, bf16) in T0's place
//     T1 = K G^T    -> rows times lam^{L-1-j};  T1 += P^T dO   -> dv out
//     T0 = dO V^T   -> P' (decayed, masked, bf16) to shared memory
//     T1 = dO S     -> dq += rows times scale lam^{i+1};       dq += P' K
//     T0 = V G      -> dk += rows times lam^{L-1-j};           dk += P'^T Q
// The row factors are applied in fp32 to the products, so that a term carries
// two bf16 roundings at most beside its inputs': of the score or of the state
// (2^-8 each).  P' in shared memory serves as both P' and P'^T.  (A first version
// with 8 epilogue warps, rounded scaled rows and P'^T as a ninth product spent
// 20,300 clocks a head, 9,200 of them in the epilogue.)
// Shared memory holds one head's tiles and P': 7 x 32 KB; the order of the
// products frees V, dO, S and G early enough for the next head's to come.
// Bound: HBM, 160 KB per chunk and v-head (V, dO, S, G, dv) and q, k, dq, dk per
// group (203 KB with three v-heads a group), against eight 128^3 products (34 MFLOP).
// Measured, 48 heads: 65,536 tokens 1,000 us, 5 TB/s (the call's 2,140 less 1,138 for
// the states); 4,096 tokens 83 us.  A head takes some 9,000 clocks, its products half
// of them: product and epilogue follow one another, and dq, dk and two working
// accumulators fill tensor memory, so that two heads cannot be in flight.  (Tried: the
// next head's first product into T1 before this one's T0 is read out, no faster; V G
// before dO S, which lets go of G and V earlier, 2% slower.  Gradients of whole chunks
// leave as tiles by TMA: rows straight from registers are a line per thread, and 13%
// more time for the kernel.)
#include "linear_tc.cuh"

namespace gdn {
namespace linear {
namespace {

constexpr int kEpiWarps = 16, kEpiThreads = 32 * kEpiWarps;
constexpr int kThreads = kEpiThreads + 64;
constexpr int kSteps = 6;  // products of a head that the epilogue works on
enum Buf { B_V = 0, B_DO, B_K, B_S, B_Q, B_G, kBufs };
constexpr uint32_t OFF_P = kBufs * kTile, OFF_MISC = OFF_P + kTile;

struct Item {
    int64_t t0;
    int32_t L, j;
};

struct Misc {
    float before[32];    // read, not used: entries -31 .. -1 of the first table
    float up[2][4][32];  // per head (in turn) and lane quarter: lam^0 .. lam^31
    uint64_t full[kBufs], empty[kBufs];
    uint64_t item_full[2], item_empty[2];
    uint64_t mma_done[kSteps], epi_done[kSteps], clean, drain;
    Item item[2];
    uint32_t tmem;
    volatile int32_t abort;
};
constexpr uint32_t kSmem = OFF_MISC + sizeof(Misc) + 1024;
static_assert(kSmem <= 232448, "shared memory of an SM");

constexpr uint32_t TM_DQ = 0, TM_DK = 128, TM_T0 = 256, TM_T1 = 384;

struct Maps {
    CUtensorMap q, k, v, g, dq, dk, dv;  // g: dO
};

// Tiles, in the order in which the head before lets go of their buffers.
__device__ void produce(const Maps &m, const BackwardPass &p, int64_t items, uint8_t *sm, Misc *ms, int G) {
    volatile int32_t *abort = &ms->abort;
    uint32_t cnt[kBufs] = {0, 0, 0, 0, 0, 0};  // loads issued into each buffer
    bool ok = true;
    auto acquire = [&](int b) {
        if (ok && cnt[b] > 0) ok = thread_wait(&ms->empty[b], (cnt[b] - 1) & 1, abort, p.err);
        if (ok) {
            ++cnt[b];
            mbar_arrive_expect_tx(&ms->full[b], kTile);
        }
        return ok;
    };
    uint32_t n = 0;
    for (int64_t it = blockIdx.x; ok && it < items; it += gridDim.x) {
        const int64_t slot = it / p.Hqk;
        const int j = (int)(it - slot * p.Hqk);
        Span sp;
        if (!find_span(p.cu, p.N, p.T, kC, slot, p.err, sp) || sp.t1 <= sp.t0) continue;
        if (n >= 2 && !(ok = thread_wait(&ms->item_empty[n & 1], ((n >> 1) - 1) & 1, abort, p.err))) break;
        ms->item[n & 1] = {sp.t0, (int32_t)(sp.t1 - sp.t0), j};
        mbar_arrive(&ms->item_full[n & 1]);
        ++n;
        for (int g = 0; g < G && ok; ++g) {
            const int h = j * G + g;
            const int64_t img = (slot * p.Hv + h) * (int64_t)kTile;
            if (g == 0) {
                if (!acquire(B_K)) break;
                load_tile(sm + B_K * kTile, &m.k, &ms->full[B_K], j, sp.t0);
                if (!acquire(B_Q)) break;
                load_tile(sm + B_Q * kTile, &m.q, &ms->full[B_Q], j, sp.t0);
            }
            if (!acquire(B_DO)) break;
            load_tile(sm + B_DO * kTile, &m.g, &ms->full[B_DO], h, sp.t0);
            if (!acquire(B_S)) break;
            bulk_load(sm + B_S * kTile, p.dump_s + img, kTile, &ms->full[B_S]);
            if (!acquire(B_G)) break;
            bulk_load(sm + B_G * kTile, p.dump_g + img, kTile, &ms->full[B_G]);
            if (!acquire(B_V)) break;
            load_tile(sm + B_V * kTile, &m.v, &ms->full[B_V], h, sp.t0);
        }
    }
    if (ok && n >= 2) ok = thread_wait(&ms->item_empty[n & 1], ((n >> 1) - 1) & 1, abort, p.err);
    if (ok) {
        ms->item[n & 1].L = -1;
        mbar_arrive(&ms->item_full[n & 1]);
        return;
    }
    // given up: let the loads in flight land before the CTA ends
    for (int b = 0; b < kBufs; ++b)
        if (cnt[b] > 0) mbar_wait_bounded(&ms->full[b], (cnt[b] - 1) & 1, kWaitLimit);
}

// Issues every MMA (one thread).  Product k of a head (0 .. 5) is handed to the
// epilogue by a commit to mma_done[k], and comes back by epi_done[k]: a barrier for
// each, because two products may be done before the first is waited for.
__device__ void multiply(const BackwardPass &p, uint32_t sbase, Misc *ms, uint32_t tmem, int G) {
    volatile int32_t *abort = &ms->abort;
    auto wait = [&](uint64_t &bar, uint32_t parity) { return thread_wait(&bar, parity & 1, abort, p.err); };
    auto tile = [&](int b) { return sbase + b * kTile; };
    const uint32_t dq = tmem + TM_DQ, dk = tmem + TM_DK, T0 = tmem + TM_T0, T1 = tmem + TM_T1;
    const uint32_t P = sbase + OFF_P;
    uint32_t u = 0, dirty = 0;  // v-heads, partial-chunk heads so far
    auto epi = [&](int k) {  // the epilogue is done with product k
        const bool ok = wait(ms->epi_done[k], u);
        tc_fence_after_sync();
        return ok;
    };
    for (uint32_t n = 0;; ++n) {
        if (!wait(ms->item_full[n & 1], n >> 1)) break;
        const int L = ms->item[n & 1].L;
        if (L < 0) {
            if (n > 0) mma_commit(&ms->mma_done[0]);  // the last item's dq and dk
            return;
        }
        mbar_arrive(&ms->item_empty[n & 1]);
        bool ok = true;
        for (int g = 0; g < G; ++g, ++u) {
            const bool last = g == G - 1;
            if (!(ok = wait(ms->full[B_K], n) && wait(ms->full[B_Q], n))) break;
            if (L < kC && !(ok = wait(ms->clean, dirty++))) break;
            mma_kk(T0, tile(B_K), tile(B_Q));
            mma_commit(&ms->mma_done[0]);
            if (!(ok = wait(ms->full[B_G], u))) break;
            mma_kk(T1, tile(B_K), tile(B_G));
            mma_commit(&ms->mma_done[1]);
            if (!(ok = wait(ms->full[B_DO], u) && epi(0) && epi(1))) break;  // P^T; scaled T1
            mma_tm(T1, T0, tile(B_DO), true);
            mma_commit(&ms->mma_done[2]);
            if (!(ok = wait(ms->full[B_V], u) && wait(ms->full[B_S], u) && epi(2))) break;  // dv out
            mma_kk(T0, tile(B_DO), tile(B_V));
            mma_commit(&ms->mma_done[3]);
            mma_km(T1, tile(B_DO), tile(B_S));
            mma_commit(&ms->empty[B_DO]);
            mma_commit(&ms->empty[B_S]);
            mma_commit(&ms->mma_done[4]);
            if (!(ok = epi(3))) break;  // P'
            mma_km(T0, tile(B_V), tile(B_G));
            mma_commit(&ms->empty[B_G]);
            mma_commit(&ms->empty[B_V]);
            mma_commit(&ms->mma_done[5]);
            if (!(ok = epi(4))) break;  // dq's first part
            mma_km(dq, P, tile(B_K), true);
            if (last) mma_commit(&ms->empty[B_K]);
            if (!(ok = epi(5))) break;  // dk's first part
            mma_mm(dk, P, tile(B_Q), true);
            if (last) mma_commit(&ms->empty[B_Q]);
        }
        if (!ok) break;
    }
    // given up: let the MMAs in flight finish before tensor memory is freed
    mma_commit(&ms->drain);
    mbar_wait_bounded(&ms->drain, 0, kWaitLimit);
}

// The 128 threads that share a quarter of the lanes.
__device__ __forceinline__ void quad_barrier(int quad) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + quad) : "memory");
}

// Whether any of the epilogue's threads has given up, the same answer for all.
__device__ __forceinline__ bool any_gave_up(bool ok) {
    uint32_t any;
    asm volatile(
        "{\n"
        ".reg .pred p, q;\n"
        "setp.eq.u32 p, %1, 0;\n"
        "barrier.cta.red.or.pred q, 5, %2, p;\n"
        "selp.u32 %0, 1, 0, q;\n"
        "}\n"
        : "=r"(any)
        : "r"((uint32_t)ok), "n"(kEpiThreads)
        : "memory");
    return any != 0;
}

// All of the epilogue's threads.
__device__ __forceinline__ void epi_barrier() { asm volatile("bar.sync 6, %0;" ::"n"(kEpiThreads) : "memory"); }

__device__ void epilogue(const Maps &m, const BackwardPass &p, uint8_t *sm, Misc *ms, uint32_t tmem, int G) {
    volatile int32_t *abort = &ms->abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, cg = warp >> 2;
    const int row = quad * 32 + lane;  // token of the chunk; columns 32 cg ..
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16), tcol = trow + 32 * cg;
    const float *up = nullptr;
    auto wait = [&](uint64_t &bar, uint32_t parity) { return warp_wait(&bar, parity & 1, abort, p.err); };
    // After a wait given up the remaining ones fail at once (abort is up), and a
    // thread goes on through its barriers: they stay whole.
    bool ok = true;
    uint32_t u = 0;  // v-heads so far
    auto product = [&](int k) {
        ok = ok && wait(ms->mma_done[k], u);
        tc_fence_after_sync();
    };
    auto done = [&](int k) {
        tmem_wait_st();
        tc_fence_before_sync();
        warp_arrive(&ms->epi_done[k]);
    };
    // this thread's 32 values of T0, times scale lam^|row - column| where the column is not
    // after (kLower) or not before the row, 0 elsewhere, as 16 words of bf16 pairs
    auto masked = [&](bool lower, float l2, uint32_t (&out)[16]) {
        float v[32];
        tmem_ld32(tcol + TM_T0, v);
        tmem_wait_ld();
        if (lower ? cg > quad : cg < quad) {
#pragma unroll
            for (int x = 0; x < 16; ++x) out[x] = 0u;
        } else if (cg != quad) {
            const float f = p.scale * exp2f(l2 * (float)(lower ? row - 32 * cg - 31 : 32 * cg - row));
            const float2 f2 = make_float2(f, f);
#pragma unroll
            for (int x = 0; x < 32; x += 4) {  // lower: lam^{31-x}, read backwards
                const float4 w = *reinterpret_cast<const float4 *>(up + (lower ? 28 - x : x));
                const float2 w0 = lower ? make_float2(w.w, w.z) : make_float2(w.x, w.y);
                const float2 w1 = lower ? make_float2(w.y, w.x) : make_float2(w.z, w.w);
                out[x / 2] = pack_bf16(fmul2(make_float2(v[x], v[x + 1]), fmul2(w0, f2)));
                out[x / 2 + 1] = pack_bf16(fmul2(make_float2(v[x + 2], v[x + 3]), fmul2(w1, f2)));
            }
        } else {
            const float *w = lower ? up + lane : up - lane;  // lam^|row - column| where it is wanted
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                const float f = p.scale * w[lower ? -x : x];
                v[x] = (lower ? x <= lane : x >= lane) ? v[x] * f : 0.f;
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) out[x] = pack_bf16(v[2 * x], v[2 * x + 1]);
        }
    };
    // this thread's 32 columns of an accumulator as 16 words of bf16 pairs, and into its token's
    // row of dst
    auto read = [&](uint32_t col, uint32_t (&w)[16]) {
        float v[32];
        tmem_ld32(tcol + col, v);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 16; ++x) w[x] = pack_bf16(v[2 * x], v[2 * x + 1]);
    };
    auto write = [&](const uint32_t (&w)[16], void *dst, int64_t t0, int L, int H, int h) {
        if (row >= L || !ok) return;
        __nv_bfloat16 *d = static_cast<__nv_bfloat16 *>(dst) + ((t0 + row) * H + h) * (int64_t)kD + 32 * cg;
#pragma unroll
        for (int c = 0; c < 16; c += 8)
            store_b256(d + 2 * c, {w[c], w[c + 1], w[c + 2], w[c + 3], w[c + 4], w[c + 5], w[c + 6], w[c + 7]});
    };
    // these 16 words of every thread to P's place, as a tile
    auto to_tile = [&](const uint32_t (&w)[16]) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4 *>(sm + OFF_P + (cg >> 1) * kSub + sw128(row, 64 * (cg & 1) + 16 * x)) =
                make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
        fence_proxy_async_smem();
    };
    // a whole chunk's tile to dst by TMA, through P's place while no P' is in it (rows from
    // registers are 64 bytes a thread, a line each, and hold up the SM's other accesses)
    auto clear_tile = [&] {
        if (tid == 0) bulk_wait_read_all();
        epi_barrier();
    };
    auto store_tile = [&](const uint32_t (&w)[16], const CUtensorMap &dst, int64_t t0, int h) {
        clear_tile();
        to_tile(w);
        epi_barrier();
        if (tid == 0 && ok) {
            tma_store_3d(&dst, sm + OFF_P, 0, h, (int32_t)t0);
            tma_store_3d(&dst, sm + OFF_P + kSub, 64, h, (int32_t)t0);
            bulk_commit();
        }
    };
    auto write_item = [&](const Item &im) {
        uint32_t w[16];
        read(TM_DQ, w);
        write(w, p.dq, im.t0, im.L, p.Hqk, im.j);
        read(TM_DK, w);
        write(w, p.dk, im.t0, im.L, p.Hqk, im.j);
    };
    // acc = (first ? 0 : acc) + f T
    auto add = [&](uint32_t acc, uint32_t T, float f, bool first) {
        const float2 f2 = make_float2(f, f);
#pragma unroll
        for (int c = 0; c < 32; c += 16) {
            float t[16], a[16];
            tmem_ld16(tcol + T + c, t);
            if (first) {
#pragma unroll
                for (int x = 0; x < 16; ++x) a[x] = 0.f;
            } else {
                tmem_ld16(tcol + acc + c, a);
            }
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; x += 2) {
                const float2 s = ffma2(f2, make_float2(t[x], t[x + 1]), make_float2(a[x], a[x + 1]));
                a[x] = s.x;
                a[x + 1] = s.y;
            }
            tmem_st16(tcol + acc + c, a);
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

    Item prev{0, -1, 0};
    for (uint32_t n = 0;; ++n) {
        ok = ok && wait(ms->item_full[n & 1], n >> 1);
        if (any_gave_up(ok)) return;
        const Item im = ms->item[n & 1];
        if (im.L < 0) break;
        warp_arrive(&ms->item_empty[n & 1]);
        for (int g = 0; g < G; ++g, ++u) {
            const int h = im.j * G + g;
            const float l2 = log2_decay(p.log_decay, h);
            if (im.L < kC) {
                ok = ok && wait(ms->full[B_V], u) && wait(ms->full[B_DO], u) && wait(ms->full[B_K], n) &&
                     wait(ms->full[B_Q], n);
                if (ok) {
                    clear(B_V, im.L);
                    clear(B_DO, im.L);
                    if (g == 0) {
                        clear(B_K, im.L);
                        clear(B_Q, im.L);
                    }
                    fence_proxy_async_smem();
                }
                warp_arrive(&ms->clean);
            }
            float *table = ms->up[u & 1][quad];
            if (cg == 0) table[lane] = exp2f(l2 * (float)lane);
            up = table;
            quad_barrier(quad);
            const float fi = p.scale * exp2f(l2 * (float)(row + 1));
            const float fj = row < im.L ? exp2f(l2 * (float)(im.L - 1 - row)) : 0.f;
            uint32_t out[16];

            product(0);  // T0 = K Q^T, and all of the previous item
            masked(false, l2, out);
            quad_barrier(quad);  // T0's rows have been read: P^T takes their place
            tmem_st16u(trow + TM_T0 + 16 * cg, out);
            done(0);
            const bool write_prev = g == 0 && prev.L == kC;
            if (write_prev) {
                read(TM_DQ, out);
                store_tile(out, m.dq, prev.t0, prev.j);
            }
            product(1);  // T1 = K G^T
            add(TM_T1, TM_T1, fj, true);
            done(1);
            if (write_prev) {
                read(TM_DK, out);
                store_tile(out, m.dk, prev.t0, prev.j);
            }
            product(2);  // T1 = dv
            read(TM_T1, out);
            done(2);
            if (im.L == kC) store_tile(out, m.dv, im.t0, h);
            else write(out, p.dv, im.t0, im.L, p.Hv, h);
            product(3);  // T0 = dO V^T
            masked(true, l2, out);
            if (write_prev || im.L == kC) clear_tile();
            to_tile(out);
            done(3);
            if (g == 0 && prev.L >= 0 && !write_prev) write_item(prev);
            product(4);  // T1 = dO S
            add(TM_DQ, TM_T1, fi, g == 0);
            done(4);
            product(5);  // T0 = V G
            add(TM_DK, TM_T0, fj, g == 0);
            done(5);
        }
        prev = im;
    }
    if (prev.L >= 0) {
        product(0);
        write_item(prev);
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
        for (int b = 0; b < kSteps; ++b) {
            mbar_init(&ms->mma_done[b], 1);
            mbar_init(&ms->epi_done[b], kEpiWarps);
        }
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
    prior_done();
    if (warp == kEpiThreads / 32) {
        if (lane == 0) produce(maps, p, items, sm, ms, G);
    } else if (warp == kEpiThreads / 32 + 1) {
        if (lane == 0) multiply(p, smem_u32(sm), ms, tmem, G);
    } else {
        epilogue(maps, p, sm, ms, tmem, G);
        if (tid == 0) bulk_wait_all();
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
        !make_tile_map_bf16_128(&m.v, p.v, p.T, p.Hv, kC) || !make_tile_map_bf16_128(&m.g, p.dO, p.T, p.Hv, kC) ||
        !make_tile_map_bf16_128(&m.dq, p.dq, p.T, p.Hqk, kC) || !make_tile_map_bf16_128(&m.dk, p.dk, p.T, p.Hqk, kC) ||
        !make_tile_map_bf16_128(&m.dv, p.dv, p.T, p.Hv, kC))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(gdn_linear_backward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmem);
    if (e != cudaSuccess) return e;
    const int64_t items = slots_of(p.T, p.N, kC) * p.Hqk, sms = device_sms();
    return launch_after(gdn_linear_backward_kernel, true, dim3((unsigned)(items < sms ? items : sms)), kThreads, kSmem, s,
                        m, p, items);
}

}  // namespace linear
}  // namespace gdn
