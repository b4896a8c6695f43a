// Linear attention with a decay per head: what its translation units share.
//
//     S_t = lam S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   lam = exp(log_decay[h])
//
// (page "Qwen3.8-27B 架构深读…", section 三, gives the undecayed sum S = sum v k^T
// read out by the query; the decay per head is the gate of the same section
// held constant.)  The forward pass and each of the three gradients are one
// form, a "pass" over arrays a, b, c with a state M (Dc x Da):
//     out_i = out_scale sum_{j <= i} lam^{i-j} (a_i . b_j) c'_j  +  the entering
//             state's part,   M += c' b^T per token,   c' = c_scale c
//     forward  a = q,  b = k,  c = v, M = S           tokens ascending
//     dq       a = do, b = v,  c = k, M = S^T         tokens ascending
//     dv       a = k,  b = q,  c = do, M = G          tokens descending
//     dk       a = v,  b = do, c = q, M = G^T         tokens descending
// with G_t = dL/dS_t = scale do_t q_t^T + lam G_{t+1}.  Ascending passes decay M
// before a token's update, descending ones after its read-out.
//
// Segments: to use the whole GPU when there are few (sequence, head) units, a
// sequence is cut into segments of seg_len tokens.  A first pass finds each
// segment's own sum from a zero state, a scan turns these into the state
// entering every segment, and the pass proper starts from it.  The host knows
// only N and T, never cu_seqlens: sequence n owns the segment slots
// [cu[n]/seg_len + n, cu[n+1]/seg_len + n + 1), at least as many as it has
// segments (ceil((b-a)/s) <= floor(b/s) - floor(a/s) + 1), T/seg_len + N in all.
#pragma once

#include <type_traits>
#include <utility>

#include "gdn_internal.cuh"
#include "sm100.cuh"

namespace gdn {
namespace linear {

// States of the sequences: array entry n, or pool slot slot[n]; a sequence with
// reset[n] set, or with a slot out of range, starts from zeros.
struct StateMap {
    const int32_t *slot = nullptr, *reset = nullptr;
    int32_t num_slots = 0;
};

struct Pass {
    const void *a, *b, *c;
    void *out;
    int32_t Ha, Hb, Hc, Hout;   // heads of each array; H of the pass
    int32_t H, Da, Dc;
    gdn_dtype dtype, out_dtype;
    const float *log_decay;     // [H]
    float c_scale, out_scale;
    bool reverse;
    const float *m0;            // [.][H][Dc][Da] entering states, or null (zeros)
    bool m0_transposed;         // m0 is [.][H][Da][Dc]
    float *mT;                  // [.][H][Dc][Da] leaving states, or null
    StateMap map;
    const int32_t *cu;
    int32_t N;
    int64_t T;
    int32_t *err;
    float *seg;                 // [seg slots][H][Dc][Da], or null: one segment per sequence
    int64_t seg_len;
};

// Kernels of one call that follow one another on its stream start early: launch_after
// lets a kernel's CTAs on to SMs as the one before it leaves them, and they wait
// (prior_done) before they touch anything that an earlier kernel of the call writes.
// Every CTA waits, those with nothing to do too, so that a kernel's end means that all
// before it have ended; and a kernel lets the next one on only once its own CTAs hold
// what they need (next_may_start).  A call's first kernel is launched plainly, and so
// are the token-recurrent ones: the wait cost their register allocation 5%.  (4,096
// tokens, 48 heads, four kernels: 115.5 us without, 107.8 with.)
__device__ __forceinline__ void prior_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), bool after, dim3 grid, int threads, size_t smem, cudaStream_t s,
                         A &&...args) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = after ? 1 : 0;
    cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
    return cudaGetLastError();
}

// First slot of sequence n among slots of `len` tokens.  (A 32-bit division, which is a
// fraction of a 64-bit one: len <= 2^31, and a negative entry of cu is found elsewhere.)
__device__ __forceinline__ int64_t slot_base(const int32_t *cu, int n, int64_t len) {
    return (int64_t)(cu ? (uint32_t)cu[n] / (uint32_t)len : 0u) + n;
}

// One segment (or chunk): tokens [t0, t1) of sequence n, number `s` of `count`.
struct Span {
    int n;
    int64_t s, count, t0, t1;
};

// The span of slot `slot`; false for a slot no segment uses, or a malformed
// cu_seqlens (reported).  Uniform across a CTA when every thread passes the
// same slot.  An empty sequence has one empty span, which carries its state.
__device__ __forceinline__ bool find_span(const int32_t *cu, int32_t N, int64_t T, int64_t len,
                                          int64_t slot, int32_t *err, Span &sp) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {  // the last n whose first slot is <= slot
        const int mid = (lo + hi + 1) >> 1;
        if (slot_base(cu, mid, len) <= slot) lo = mid;
        else hi = mid - 1;
    }
    int64_t b, e;
    if (!seq_range(cu, lo, N, T, err, b, e)) return false;
    sp.n = lo;
    // 0 <= b <= e <= T < 2^31
    sp.s = slot - ((int64_t)((uint32_t)b / (uint32_t)len) + lo);
    sp.count = e > b ? (int64_t)((uint32_t)(e - b - 1) / (uint32_t)len) + 1 : 1;
    if (sp.s < 0 || sp.s >= sp.count) return false;
    sp.t0 = b + sp.s * len;
    sp.t1 = sp.t0 + len < e ? sp.t0 + len : e;
    return true;
}

// Whatever the slots of a malformed cu_seqlens map to, each of its ranges is
// looked at (and reported) by the CTAs of one slot, in a warp that is not first
// to work: slots >= N.
__device__ __forceinline__ void check_range(const int32_t *cu, int32_t N, int64_t T, int64_t slot, int32_t *err) {
    int64_t b, e;
    if (cu != nullptr && slot < N) seq_range(cu, (int)slot, N, T, err, b, e);
}

inline int64_t slots_of(int64_t T, int32_t N, int64_t len) { return T / len + N; }

// Index of sequence n's state, or -1 (a slot out of range).
__device__ __forceinline__ int64_t state_index(const StateMap &m, int n) {
    if (m.slot == nullptr) return n;
    const int s = m.slot[n];
    return s >= 0 && s < m.num_slots ? s : -1;
}
__device__ __forceinline__ bool state_fresh(const StateMap &m, int n) {
    return m.reset != nullptr && m.reset[n] != 0;
}

// The decay exp(g) of a token, chunk or segment, applied to fp32 values.  A slow one acts
// many times, so its own rounding must not: x + x expm1(g) keeps 24 bits of 1 - lam.  A
// strong one is a plain product, which keeps 24 bits of lam.  (With a rounded factor near
// 1, the same at every chunk, final states were off by 3.2e-5 after 513 chunks at
// log_decay near -1e-6, and in proportion to their number; now by less than 2.8e-6.)
struct Decay {
    float f;
    bool slow;
    __device__ __forceinline__ explicit Decay(float g) : slow(g > -0.5f) { f = slow ? expm1f(g) : expf(g); }
    template <bool kSlow>
    __device__ __forceinline__ float times(float x) const {
        return kSlow ? fmaf(f, x, x) : f * x;
    }
    template <bool kSlow>
    __device__ __forceinline__ float2 times(float2 x) const {
        const float2 f2 = make_float2(f, f);
        return kSlow ? sm100::ffma2(f2, x, x) : sm100::fmul2(f2, x);
    }
    // exp(g) x + y
    template <bool kSlow>
    __device__ __forceinline__ float2 plus(float2 x, float2 y) const {
        const float2 z = sm100::ffma2(make_float2(f, f), x, y);
        return kSlow ? sm100::ffma2(make_float2(1.f, 1.f), x, z) : z;
    }
};

// Token-recurrent passes for any Da, Dc of 16, 32, 64, 128 and either dtype.
// `phase` 0: the whole pass; 1: the segments' own sums into p.seg.
cudaError_t launch_recurrent(const Pass &p, int phase, cudaStream_t s);
// The states entering every segment, in place of the sums in p.seg; of one pass, or of
// two of the same N, H, Da and Dc.
cudaError_t launch_scan(const Pass *p, int passes, cudaStream_t s);
// Segment length for the recurrent passes, or 0 for one segment per sequence.
int64_t recurrent_seg_len(int32_t N, int64_t T, int32_t H, int32_t Da, int32_t Dc);
// dst[t][j] = sum of the H / Hout heads of group j, in dst's dtype.
cudaError_t launch_group_sum(const float *src, void *dst, gdn_dtype dt, int64_t T, int32_t H,
                             int32_t Hout, int32_t D, cudaStream_t s);

struct DecodeStep {
    const void *q, *k, *v;
    void *o;
    gdn_dtype dtype;
    const float *log_decay;
    float scale;
    float *state;
    StateMap map;
    int32_t N, Hqk, Hv, Dk, Dv;
    int32_t *err;
};
cudaError_t launch_decode(const DecodeStep &d, cudaStream_t s);

}  // namespace linear
}  // namespace gdn
