// C entry points of linear attention with a decay per head: argument
// validation and dispatch (include/gdn.h has the contracts).
#include "linear_tc.cuh"
#include "trace.cuh"

namespace {

using gdn::linear::Pass;
using gdn::linear::StateMap;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool supported_dim(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }
gdn_status from_cuda(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }
size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// What gdn_linear_prefill, its slot form and its backward pass have in common.
struct Call {
    gdn_dtype dt;
    const int32_t *cu;
    int32_t N;
    int64_t T;
    int32_t Hqk, Hv, Dk, Dv;
};

gdn_status check(const Call &c) {
    if (c.dt != GDN_DTYPE_BF16 && c.dt != GDN_DTYPE_F32) return GDN_ERR_INVALID_ARGUMENT;
    if (c.N < 0 || c.T < 0 || c.Hqk <= 0 || c.Hv <= 0 || c.Dk <= 0 || c.Dv <= 0)
        return GDN_ERR_INVALID_ARGUMENT;
    if (c.Hv % c.Hqk != 0) return GDN_ERR_INVALID_ARGUMENT;
    if (c.cu == nullptr && c.N != 1) return GDN_ERR_INVALID_ARGUMENT;
    if (c.N == 0 && c.T != 0) return GDN_ERR_INVALID_ARGUMENT;
    return GDN_OK;
}

gdn_status check_size(const Call &c) {
    if (!supported_dim(c.Dk) || !supported_dim(c.Dv)) return GDN_ERR_UNSUPPORTED;
    // token indices are 32-bit in cu_seqlens and in TMA coordinates, and the
    // largest grid has (T / 128 + N + 1) * Hv * 4 CTAs (divided: the product can pass 64 bits)
    if (c.T > 0x7fffffffLL || c.T / 128 + c.N + 1 > 0x7fffffffLL / 4 / c.Hv) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

template <int NP, int NI, int NO>
gdn_status check_pointers(const void *const (&all)[NP], const void *const (&ins)[NI],
                          const void *const (&outs)[NO]) {
    for (const void *p : all)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < NO; ++i) {
        for (const void *in : ins)
            if (outs[i] && outs[i] == in) return GDN_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (outs[i] && outs[i] == outs[j]) return GDN_ERR_INVALID_ARGUMENT;
    }
    return GDN_OK;
}

size_t seg_bytes(const Call &c, int64_t seg_len) {
    return seg_len ? al256((size_t)gdn::linear::slots_of(c.T, c.N, seg_len) * c.Hv * c.Dk * c.Dv * 4) : 0;
}

// The tensor-core kernels serve 128-wide bf16 heads, from `least` tokens a sequence on
// average: below that a token at a time is faster than 128-token chunks.  (48 heads, a
// token at a time and on tensor cores: prefill of 64 sequences of 16 tokens 293 and 290
// us, of 24 393 and 291, of 8 sequences of 12 32 and 44; gradients of 64 sequences of 4
// tokens 638 and 570, of 8 98 and 81, of one 41 and 33.)
constexpr int kLeastPrefill = 16, kLeastBackward = 2;
bool tensor_cores(const Call &c, int least) {
    return c.dt == GDN_DTYPE_BF16 && c.Dk == 128 && c.Dv == 128 && c.T > (int64_t)least * c.N;
}

size_t prefill_bytes(const Call &c) {
    if (check(c) != GDN_OK || check_size(c) != GDN_OK || c.T == 0) return 0;
    if (tensor_cores(c, kLeastPrefill))
        return gdn::linear::state_dump_bytes(c.N, c.T, c.Hv) + gdn::linear::state_seg_bytes(c.N, c.T, c.Hv, 1);
    return seg_bytes(c, gdn::linear::recurrent_seg_len(c.N, c.T, c.Hv, c.Dk, c.Dv));
}

// Tensor cores: the images of S and of G, and the segment states of each.
// Otherwise the three gradients run one after another and share the segment
// states; dq and dk of v-heads that share a q/k head are summed from fp32 partials.
size_t backward_bytes(const Call &c) {
    if (check(c) != GDN_OK || check_size(c) != GDN_OK || c.T == 0) return 0;
    if (tensor_cores(c, kLeastBackward))
        return 2 * gdn::linear::state_dump_bytes(c.N, c.T, c.Hv) + 2 * gdn::linear::state_seg_bytes(c.N, c.T, c.Hv, 2);
    const size_t a = seg_bytes(c, gdn::linear::recurrent_seg_len(c.N, c.T, c.Hv, c.Dk, c.Dv));
    const size_t b = seg_bytes(c, gdn::linear::recurrent_seg_len(c.N, c.T, c.Hv, c.Dv, c.Dk));
    const size_t part = c.Hv > c.Hqk ? al256((size_t)c.T * c.Hv * c.Dk * 4) : 0;
    return (a > b ? a : b) + part;
}

// A pass with its segments (p.seg is the workspace for them).
cudaError_t run(Pass p, void *ws, cudaStream_t s) {
    p.seg_len = gdn::linear::recurrent_seg_len(p.N, p.T, p.H, p.Da, p.Dc);
    p.seg = p.seg_len ? static_cast<float *>(ws) : nullptr;
    if (p.seg) {
        cudaError_t e = gdn::linear::launch_recurrent(p, 1, s);
        if (e == cudaSuccess) e = gdn::linear::launch_scan(&p, 1, s);
        if (e != cudaSuccess) return e;
    }
    return gdn::linear::launch_recurrent(p, 0, s);
}

// State pass `which` of `passes` that run together: the workspace holds their image
// arrays, then their segment states.
gdn::linear::StatePass states(const Call &c, const void *x, const void *y, int32_t Hy, const float *log_decay,
                              float x_scale, bool reverse, const float *m0, float *mT, void *ws, int which,
                              int passes, int32_t *err) {
    gdn::linear::StatePass st{};
    st.x = x; st.y = y; st.H = c.Hv; st.Hy = Hy; st.log_decay = log_decay; st.x_scale = x_scale;
    st.reverse = reverse; st.m0 = m0; st.mT = mT; st.cu = c.cu; st.N = c.N; st.T = c.T; st.err = err;
    const size_t dump = gdn::linear::state_dump_bytes(c.N, c.T, c.Hv);
    uint8_t *base = static_cast<uint8_t *>(ws);
    st.dump = base + which * dump;
    st.seg_chunks = gdn::linear::state_seg_chunks(c.N, c.T, c.Hv, passes);
    if (st.seg_chunks)
        st.seg = reinterpret_cast<float *>(base + passes * dump +
                                           which * gdn::linear::state_seg_bytes(c.N, c.T, c.Hv, passes));
    return st;
}

gdn_status prefill(const void *q, const void *k, const void *v, const float *log_decay, float scale,
                   const float *s0, float *sT, const StateMap &map, const Call &c, void *o, void *ws,
                   size_t ws_bytes, int32_t *err, cudaStream_t s) {
    const size_t need = prefill_bytes(c);
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return GDN_ERR_INVALID_ARGUMENT;
    if (c.N == 0 || (c.T == 0 && sT == nullptr)) return GDN_OK;  // nothing observable to do
    if (tensor_cores(c, kLeastPrefill)) {
        gdn::linear::StatePass st = states(c, v, k, c.Hqk, log_decay, 1.f, false, s0, sT, ws, 0, 1, err);
        st.map = map;
        const cudaError_t e = gdn::linear::launch_states(&st, 1, s);
        if (e != cudaSuccess) return from_cuda(e);
        return from_cuda(gdn::linear::launch_out({q, k, v, o, st.dump, log_decay, scale, c.cu, c.N, c.T, c.Hqk,
                                                  c.Hv, err}, s));
    }
    Pass p{};
    p.a = q; p.b = k; p.c = v; p.out = o;
    p.Ha = c.Hqk; p.Hb = c.Hqk; p.Hc = c.Hv; p.Hout = c.Hv; p.H = c.Hv; p.Da = c.Dk; p.Dc = c.Dv;
    p.dtype = c.dt; p.out_dtype = c.dt;
    p.log_decay = log_decay; p.c_scale = 1.f; p.out_scale = scale;
    p.m0 = s0; p.mT = sT; p.map = map;
    p.cu = c.cu; p.N = c.N; p.T = c.T; p.err = err;
    return from_cuda(run(p, ws, s));
}

}  // namespace

extern "C" {

size_t gdn_linear_prefill_workspace_bytes(int32_t N, int64_t T, int32_t Hqk, int32_t Hv, int32_t Dk,
                                          int32_t Dv, gdn_dtype io_dtype) {
    static const int32_t some = 0;
    return prefill_bytes({io_dtype, &some, N, T, Hqk, Hv, Dk, Dv});
}

size_t gdn_linear_prefill_backward_workspace_bytes(int32_t N, int64_t T, int32_t Hqk, int32_t Hv,
                                                   int32_t Dk, int32_t Dv, gdn_dtype io_dtype) {
    static const int32_t some = 0;
    return backward_bytes({io_dtype, &some, N, T, Hqk, Hv, Dk, Dv});
}

gdn_status gdn_linear_prefill(const void *q, const void *k, const void *v, gdn_dtype io_dtype,
                              const float *log_decay, float scale, const float *initial_state,
                              const int32_t *cu_seqlens, int32_t N, int64_t T, int32_t Hqk,
                              int32_t Hv, int32_t Dk, int32_t Dv, void *o, float *final_state,
                              void *workspace, size_t workspace_bytes, int32_t *dev_error_flag,
                              void *stream) {
    GDN_TRACE("gdn_linear_prefill");
    const Call c{io_dtype, cu_seqlens, N, T, Hqk, Hv, Dk, Dv};
    if (gdn_status e = check(c)) return e;
    if (T > 0 && (!q || !k || !v || !log_decay || !o)) return GDN_ERR_INVALID_ARGUMENT;
    if (N > 0 && final_state && !log_decay) return GDN_ERR_INVALID_ARGUMENT;
    const void *all[] = {q, k, v, log_decay, initial_state, cu_seqlens, o, final_state, workspace,
                         dev_error_flag};
    const void *ins[] = {q, k, v, log_decay};
    const void *outs[] = {o, final_state, workspace};
    if (gdn_status e = check_pointers(all, ins, outs)) return e;
    if (o && o == initial_state) return GDN_ERR_INVALID_ARGUMENT;
    if (gdn_status e = check_size(c)) return e;
    return prefill(q, k, v, log_decay, scale, initial_state, final_state, StateMap{}, c, o, workspace,
                   workspace_bytes, dev_error_flag, static_cast<cudaStream_t>(stream));
}

gdn_status gdn_linear_prefill_slots(const void *q, const void *k, const void *v, gdn_dtype io_dtype,
                                    const float *log_decay, float scale, float *state_pool,
                                    int32_t num_slots, const int32_t *slot_idx, const int32_t *reset,
                                    const int32_t *cu_seqlens, int32_t N, int64_t T, int32_t Hqk,
                                    int32_t Hv, int32_t Dk, int32_t Dv, void *o, void *workspace,
                                    size_t workspace_bytes, int32_t *dev_error_flag, void *stream) {
    GDN_TRACE("gdn_linear_prefill_slots");
    const Call c{io_dtype, cu_seqlens, N, T, Hqk, Hv, Dk, Dv};
    if (gdn_status e = check(c)) return e;
    if (T > 0 && (!q || !k || !v || !o)) return GDN_ERR_INVALID_ARGUMENT;
    if (N > 0 && (!log_decay || !state_pool || !slot_idx || num_slots <= 0)) return GDN_ERR_INVALID_ARGUMENT;
    const void *all[] = {q, k, v, log_decay, state_pool, slot_idx, reset, cu_seqlens, o, workspace,
                         dev_error_flag};
    const void *ins[] = {q, k, v, log_decay};
    const void *outs[] = {o, state_pool, workspace};
    if (gdn_status e = check_pointers(all, ins, outs)) return e;
    if (gdn_status e = check_size(c)) return e;
    return prefill(q, k, v, log_decay, scale, state_pool, state_pool, StateMap{slot_idx, reset, num_slots},
                   c, o, workspace, workspace_bytes, dev_error_flag, static_cast<cudaStream_t>(stream));
}

gdn_status gdn_linear_prefill_backward(const void *dO, const void *q, const void *k, const void *v,
                                       gdn_dtype io_dtype, const float *log_decay, float scale,
                                       const float *initial_state, const float *dfinal_state,
                                       const int32_t *cu_seqlens, int32_t N, int64_t T, int32_t Hqk,
                                       int32_t Hv, int32_t Dk, int32_t Dv, void *dq, void *dk, void *dv,
                                       float *dinitial_state, void *workspace, size_t workspace_bytes,
                                       int32_t *dev_error_flag, void *stream) {
    GDN_TRACE("gdn_linear_prefill_backward");
    const Call c{io_dtype, cu_seqlens, N, T, Hqk, Hv, Dk, Dv};
    if (gdn_status e = check(c)) return e;
    if (T > 0 && (!dO || !q || !k || !v || !dq || !dk || !dv)) return GDN_ERR_INVALID_ARGUMENT;
    if ((T > 0 || (N > 0 && dinitial_state)) && !log_decay) return GDN_ERR_INVALID_ARGUMENT;
    const void *all[] = {dO, q, k, v, log_decay, initial_state, dfinal_state, cu_seqlens, dq, dk, dv,
                         dinitial_state, workspace, dev_error_flag};
    const void *ins[] = {dO, q, k, v, log_decay, initial_state};
    const void *outs[] = {dq, dk, dv, dinitial_state, workspace};
    if (gdn_status e = check_pointers(all, ins, outs)) return e;
    const void *rest[] = {dq, dk, dv, workspace};
    for (const void *x : rest)
        if (x && x == dfinal_state) return GDN_ERR_INVALID_ARGUMENT;
    if (gdn_status e = check_size(c)) return e;
    const size_t need = backward_bytes(c);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return GDN_ERR_INVALID_ARGUMENT;
    if (N == 0 || (T == 0 && dinitial_state == nullptr)) return GDN_OK;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tensor_cores(c, kLeastBackward)) {
        // S and G do not depend on one another: one launch for both
        const gdn::linear::StatePass sg[2] = {states(c, v, k, Hqk, log_decay, 1.f, false, initial_state, nullptr,
                                                     workspace, 0, 2, dev_error_flag),
                                              states(c, dO, q, Hqk, log_decay, scale, true, dfinal_state,
                                                     dinitial_state, workspace, 1, 2, dev_error_flag)};
        cudaError_t e = gdn::linear::launch_states(sg, 2, s);
        if (e == cudaSuccess)
            e = gdn::linear::launch_backward({dO, q, k, v, dq, dk, dv, sg[0].dump, sg[1].dump, log_decay, scale,
                                              cu_seqlens, N, T, Hqk, Hv, dev_error_flag}, s);
        return from_cuda(e);
    }
    const bool shared = Hv > Hqk;
    const size_t part = shared ? al256((size_t)T * Hv * Dk * 4) : 0;
    float *partial = static_cast<float *>(workspace);
    void *seg = static_cast<uint8_t *>(workspace) + part;
    Pass p{};
    p.H = Hv; p.dtype = io_dtype; p.log_decay = log_decay;
    p.cu = cu_seqlens; p.N = N; p.T = T; p.err = dev_error_flag;
    auto pass = [&](const void *a, int32_t Ha, const void *b, int32_t Hb, const void *cc, int32_t Hc,
                    int32_t Da, int32_t Dc, void *out, bool sum) -> cudaError_t {
        p.a = a; p.b = b; p.c = cc; p.Ha = Ha; p.Hb = Hb; p.Hc = Hc; p.Da = Da; p.Dc = Dc;
        p.Hout = Hv;
        p.out = sum ? partial : out;
        p.out_dtype = sum ? GDN_DTYPE_F32 : io_dtype;
        cudaError_t e = run(p, seg, s);
        if (e == cudaSuccess && sum)
            e = gdn::linear::launch_group_sum(partial, out, io_dtype, T, Hv, Hqk, Dc, s);
        return e;
    };
    cudaError_t e = cudaSuccess;
    p.reverse = false; p.c_scale = 1.f; p.out_scale = scale;
    p.m0 = initial_state; p.m0_transposed = true; p.mT = nullptr;
    if (T > 0) e = pass(dO, Hv, v, Hv, k, Hqk, Dv, Dk, dq, shared);
    p.reverse = true; p.c_scale = scale; p.out_scale = 1.f;
    p.m0 = dfinal_state;
    if (e == cudaSuccess && T > 0) e = pass(v, Hv, dO, Hv, q, Hqk, Dv, Dk, dk, shared);
    // last: dinitial_state may be dfinal_state's memory
    p.m0_transposed = false; p.mT = dinitial_state;
    if (e == cudaSuccess) e = pass(k, Hqk, q, Hqk, dO, Hv, Dk, Dv, dv, false);
    return from_cuda(e);
}

}  // extern "C"

namespace {

gdn_status decode(const void *q, const void *k, const void *v, gdn_dtype io_dtype, const float *log_decay,
                  float scale, float *state, const StateMap &map, int32_t N, int32_t Hqk, int32_t Hv,
                  int32_t Dk, int32_t Dv, void *o, int32_t *err, void *stream) {
    if (io_dtype != GDN_DTYPE_BF16 && io_dtype != GDN_DTYPE_F32) return GDN_ERR_INVALID_ARGUMENT;
    if (N < 0 || Hqk <= 0 || Hv <= 0 || Dk <= 0 || Dv <= 0 || Hv % Hqk != 0) return GDN_ERR_INVALID_ARGUMENT;
    if (N > 0 && (!q || !k || !v || !log_decay || !state || !o)) return GDN_ERR_INVALID_ARGUMENT;
    const void *all[] = {q, k, v, log_decay, state, map.slot, map.reset, o, err};
    const void *ins[] = {q, k, v, log_decay};
    const void *outs[] = {o, state};
    if (gdn_status e = check_pointers(all, ins, outs)) return e;
    if (!supported_dim(Dk) || Dv > 1 << 30) return GDN_ERR_UNSUPPORTED;
    // a grid of one CTA per (sequence, v-head), or per 128 state rows of it where Dk = 128
    if ((int64_t)N * Hv > 0x7fffffffLL / (Dk == 128 ? (Dv + 127) / 128 : 1)) return GDN_ERR_UNSUPPORTED;
    if (N == 0) return GDN_OK;
    return from_cuda(gdn::linear::launch_decode({q, k, v, o, io_dtype, log_decay, scale, state, map, N, Hqk,
                                                 Hv, Dk, Dv, err},
                                                static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

gdn_status gdn_linear_decode_step(const void *q, const void *k, const void *v, gdn_dtype io_dtype,
                                  const float *log_decay, float scale, float *state, int32_t N,
                                  int32_t Hqk, int32_t Hv, int32_t Dk, int32_t Dv, void *o,
                                  int32_t *dev_error_flag, void *stream) {
    GDN_TRACE("gdn_linear_decode_step");
    return decode(q, k, v, io_dtype, log_decay, scale, state, StateMap{}, N, Hqk, Hv, Dk, Dv, o,
                  dev_error_flag, stream);
}

gdn_status gdn_linear_decode_step_slots(const void *q, const void *k, const void *v, gdn_dtype io_dtype,
                                        const float *log_decay, float scale, float *state_pool,
                                        int32_t num_slots, const int32_t *slot_idx, const int32_t *reset,
                                        int32_t N, int32_t Hqk, int32_t Hv, int32_t Dk, int32_t Dv,
                                        void *o, int32_t *dev_error_flag, void *stream) {
    GDN_TRACE("gdn_linear_decode_step_slots");
    if (N > 0 && (!slot_idx || num_slots <= 0)) return GDN_ERR_INVALID_ARGUMENT;
    return decode(q, k, v, io_dtype, log_decay, scale, state_pool, StateMap{slot_idx, reset, num_slots}, N,
                  Hqk, Hv, Dk, Dv, o, dev_error_flag, stream);
}

}  // extern "C"
