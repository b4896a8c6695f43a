// What the tensor-core kernels of linear attention share (Dk = Dv = 128, bf16,
// chunks of 128 tokens): tile constants, descriptors, bounded waits.
#pragma once

#include <cuda_bf16.h>

#include "linear.cuh"
#include "sm100.cuh"

namespace gdn {

// [T][H][128] bf16 tensor map with 64 x 1 x `rows` boxes and the 128-byte
// swizzle (rows past T read as zeros).
bool make_tile_map_bf16_128(CUtensorMap *m, const void *base, int64_t T, int32_t H, int32_t rows);

namespace linear {

using namespace sm100;

constexpr int kC = 128;                  // chunk length
constexpr int kD = 128;                  // Dk = Dv
constexpr uint32_t kSub = 16384;         // 128 rows x 64 columns of a tile, 128-byte swizzle
constexpr uint32_t kTile = 2 * kSub;     // 128 x 128 bf16
constexpr long long kWaitLimit = 1ll << 31;  // SM clocks (about a second)
constexpr float kLog2e = 1.4426950408889634f;

// bf16 operands, M = N = 128; letters: A then B, K-major or MN-major.
constexpr uint32_t IDESC_KK = make_idesc_f16(128, 128, 0, 0, 1);
constexpr uint32_t IDESC_KM = make_idesc_f16(128, 128, 0, 1, 1);
constexpr uint32_t IDESC_MM = make_idesc_f16(128, 128, 1, 1, 1);

// Descriptors of a tile stored [128 rows][128 columns]: rows are the operand's M
// (or N) index and columns the summed one (K-major), or the other way round
// (MN-major, `sub` bytes between its 64-column halves).  Step ks, 16 of the
// summed elements, is a constant further in the address field, which is all that
// an MMA's one issuing thread has to add (building each descriptor anew took it
// longer than the tensor core took for the product).
__device__ __forceinline__ uint64_t desc_k(uint32_t tile) { return make_sdesc(tile, 16, 1024); }
__device__ __forceinline__ uint64_t desc_m(uint32_t tile, uint32_t sub = kSub) {
    return make_sdesc(tile, sub, 1024);
}
__device__ __forceinline__ uint64_t step_k(uint64_t d, int ks) {
    return d + (uint64_t)(((ks >> 2) * kSub + (ks & 3) * 32) >> 4);
}
__device__ __forceinline__ uint64_t step_m(uint64_t d, int ks) { return d + (uint64_t)(ks * 2048 >> 4); }

// D (+)= A B over 128 summed elements, operands in shared memory; letters as above.
__device__ __forceinline__ void mma_kk(uint32_t d, uint32_t a, uint32_t b, bool acc = false) {
    const uint64_t da = desc_k(a), db = desc_k(b);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) mma_f16_ss(d, step_k(da, ks), step_k(db, ks), IDESC_KK, acc || ks);
}
__device__ __forceinline__ void mma_km(uint32_t d, uint32_t a, uint32_t b, bool acc = false) {
    const uint64_t da = desc_k(a), db = desc_m(b);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) mma_f16_ss(d, step_k(da, ks), step_m(db, ks), IDESC_KM, acc || ks);
}
__device__ __forceinline__ void mma_mm(uint32_t d, uint32_t a, uint32_t b, bool acc = false) {
    const uint64_t da = desc_m(a), db = desc_m(b);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) mma_f16_ss(d, step_m(da, ks), step_m(db, ks), IDESC_MM, acc || ks);
}
// A from tensor memory (K-major, 64 columns of packed pairs), B MN-major.
__device__ __forceinline__ void mma_tm(uint32_t d, uint32_t a_tmem, uint32_t b, bool acc = false) {
    const uint64_t db = desc_m(b);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) mma_f16_ts(d, a_tmem + 8 * ks, step_m(db, ks), IDESC_KM, acc || ks);
}

// 32 bytes in one access, a whole memory sector per thread, where the address is
// a multiple of 32 (the caller's arrays are multiples of 16).
__device__ __forceinline__ void store_b256(void *p, const uint32_t (&v)[8]) {
    if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
                     "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        static_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
__device__ __forceinline__ void load_b256(const void *p, uint32_t (&v)[8]) {
    if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "l"(p)
                     : "memory");
    } else {
        const uint4 a = static_cast<const uint4 *>(p)[0], b = static_cast<const uint4 *>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

// A head's log2(lam), no further down than where every power of it but the 0th is
// zero in fp32 anyway: infinity times no tokens must not arise.
__device__ __forceinline__ float log2_decay(const float *log_decay, int h) {
    const float x = log_decay[h] * kLog2e;
    return x < -1000.f ? -1000.f : x;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&t);
}
__device__ __forceinline__ uint32_t pack_bf16(float2 a) { return pack_bf16(a.x, a.y); }

// Both 64-column halves of the 128-token tile of head h at token t0.
__device__ __forceinline__ void load_tile(void *dst, const CUtensorMap *map, uint64_t *bar, int h, int64_t t0) {
    tma_load_3d(dst, map, bar, 0, h, (int32_t)t0);
    tma_load_3d(static_cast<uint8_t *>(dst) + kSub, map, bar, 64, h, (int32_t)t0);
}

// Waits of the warp-specialised kernels: give up when another role has
// (`abort`), or after kWaitLimit clocks, raising `abort` and the error flag.
// thread_wait is for the roles of one thread; the lanes of a warp may get different
// answers from it (the barrier completes for one as `abort` goes up for another).
// (A suspend-time hint on the wait made the whole chunk-state kernel 10% slower:
// the hardware wakes such a warp later.)
__device__ __forceinline__ bool thread_wait(uint64_t *bar, uint32_t parity, volatile int32_t *abort, int32_t *err) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (clock64() - t0 > kWaitLimit) {
            *abort = 1;
            raise_error(err, GDN_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
// The same for the roles of whole warps: one answer for all 32 lanes, so that none leaves
// while others go on to an instruction that needs all of them.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int32_t *abort, int32_t *err) {
    return __all_sync(0xffffffffu, thread_wait(bar, parity, abort, err));
}

// One arrival for a warp whose lanes have done their part (and fenced it): 32
// lanes arriving one by one would be 32 atomics on one word.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Two bf16 of a word as floats.
__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// The states entering every chunk, found by one pass over a value-like array x
// [T][H][128] and a key-like one y [T][Hy][128]:
//   ascending   M' = lam^L M + sum_j lam^{L-1-j} x_j y_j^T       (S: x = v, y = k)
//   descending  M' = lam^L M + x_scale sum_j lam^{j+1} x_j y_j^T  (G: x = do, y = q)
// over chunks of L <= 128 tokens.  Every chunk's entering M goes, rounded to
// bf16, to `dump` as the shared-memory image of a 128 x 128 tile (32 KB per
// (chunk slot, head)); the last M in fp32 to mT.
struct StatePass {
    const void *x, *y;
    int32_t H, Hy;
    const float *log_decay;
    float x_scale;
    bool reverse;
    const float *m0;
    float *mT;
    StateMap map;
    const int32_t *cu;
    int32_t N;
    int64_t T;
    int32_t *err;
    float *seg;          // [seg slots][H][128][128] or null
    int64_t seg_chunks;  // chunks per segment
    uint8_t *dump;
};

// Workspace of a StatePass besides its dump, of `passes` that run together; the dump's bytes.
int64_t state_seg_chunks(int32_t N, int64_t T, int32_t H, int passes);  // 0: one segment per sequence
size_t state_seg_bytes(int32_t N, int64_t T, int32_t H, int passes);    // of each pass
size_t state_dump_bytes(int32_t N, int64_t T, int32_t H);
// Runs one pass, or two of the same N, T, H, cu and seg_chunks side by side (segment
// sums and scan first when seg is set).
cudaError_t launch_states(const StatePass *p, int passes, cudaStream_t s);

struct OutPass {
    const void *q, *k, *v;
    void *o;
    const uint8_t *dump;  // S entering every chunk
    const float *log_decay;
    float scale;
    const int32_t *cu;
    int32_t N;
    int64_t T;
    int32_t Hqk, Hv;
    int32_t *err;
};
cudaError_t launch_out(const OutPass &p, cudaStream_t s);

struct BackwardPass {
    const void *dO, *q, *k, *v;
    void *dq, *dk, *dv;
    const uint8_t *dump_s, *dump_g;  // S entering and G leaving every chunk
    const float *log_decay;
    float scale;
    const int32_t *cu;
    int32_t N;
    int64_t T;
    int32_t Hqk, Hv;
    int32_t *err;
};
cudaError_t launch_backward(const BackwardPass &p, cudaStream_t s);

int device_sms();

}  // namespace linear
}  // namespace gdn
