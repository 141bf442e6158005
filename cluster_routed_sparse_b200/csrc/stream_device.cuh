// stream_device.cuh -- device helpers shared by the streaming operators (axial
// rotary embedding, window attention, 8-bit cache): strided views, the visible
// key range of a query row, e4m3 conversions and the operators' error words.
#pragma once

#include <cuda_fp16.h>

#include "ac_device.cuh"
#include "stream_internal.h"

namespace ac {

// ------------------------------------------------------------------ visible keys
// Query row i of a sequence with ql queries and kl keys stands at position
// i + kl - ql.  With blk(x) = floor(x / g), it sees key j when j < kl,
// blk(j) <= blk(pos) + right, and blk(j) >= blk(pos) - left or j < sinks: the
// union of [lo, hi) and [0, min(sinks, hi)).
struct RowRange {
    int lo, hi;
};

__device__ __forceinline__ int floor_div(int a, int g) {
    const int q = a / g;
    return q - (a % g < 0 ? 1 : 0);
}

__device__ __forceinline__ RowRange row_range(const WinRule &w, int pos, int kl) {
    const int b = w.g == 1 ? pos : floor_div(pos, w.g);
    long long lo = w.left < 0 ? 0 : ((long long)b - w.left) * w.g;
    long long hi = w.right < 0 ? kl : ((long long)b + w.right + 1) * w.g;
    hi = hi < 0 ? 0 : hi > kl ? kl : hi;
    lo = lo < 0 ? 0 : lo > hi ? hi : lo;
    return RowRange{(int)lo, (int)hi};
}

// Lengths come from device memory: out of [0, most] they are clamped and noted.
__device__ __forceinline__ int seq_len(const int *lens, int b, int most, OpErr *err) {
    if (!lens) return most;
    const int n = lens[b];
    if (n < 0 || n > most) atomicOr(&err->bits, DEV_ERR_BOUNDS);
    return n < 0 ? 0 : n > most ? most : n;
}

// Bounded wait of a launch's kernels.  The first to expire notes the launch, which ends the
// others' waits early.  What is in flight when a wait gives up is waited for with mbar_wait,
// which does not look at that note: loads and products issued end by themselves.
__device__ __forceinline__ bool wait_or_note(uint32_t bar, uint32_t parity, uint32_t *noted, uint32_t launch,
                                             uint64_t limit_ns = kWaitLimitNs) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    const long long c0 = clock64(), limit_cycles = (long long)limit_ns * 2;
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 255u) == 255u) {
            if (*reinterpret_cast<const volatile uint32_t *>(noted) == launch) return false;
            if (globaltimer_ns() - t0 > limit_ns || clock64() - c0 > limit_cycles || it > kWaitLimitPolls) {
                *reinterpret_cast<volatile uint32_t *>(noted) = launch;
                return false;
            }
        }
    }
}

// 5-D tiled bulk tensor load (coordinates x innermost).  No cluster multicast.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void *tmap, int32_t x, int32_t y, int32_t z, int32_t w,
                                            int32_t v, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar)
        : "memory");
}

// ------------------------------------------------------------------ chained launches
// A kernel that launch_after started may begin while its predecessor's last CTAs run.
// It waits here, until all of the predecessor is done and seen (the fence: by the bulk
// loads too), before it touches what this call's kernels write.
__device__ __forceinline__ void wait_predecessor() {
    asm volatile("griddepcontrol.wait;\n\tfence.proxy.async;" ::: "memory");
}
// Lets the successor's CTAs take the SMs that are free once every CTA here has begun.
__device__ __forceinline__ void release_successor() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------------ products
// The issuing warp stays converged and its descriptors are the same in every
// lane, so that they live in uniform registers; one elected lane executes the
// instruction.  (A branch to a single lane costs moves to uniform registers for
// every operand of every product: 3,500 cycles of issue per pair of 128-key tiles
// instead of the 2,048 that the products take.)
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

struct Desc {  // shared-memory matrix descriptor; offsets in 16-byte units stay within the low word
    uint32_t lo, hi;
};
__device__ __forceinline__ Desc make_desc(uint64_t d) { return Desc{(uint32_t)d, (uint32_t)(d >> 32)}; }

// D[tmem] (+)= A[smem] B[smem]^T, one K16 step
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, Desc a, Desc b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 e, %7, 0;\n\t"
        "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
        "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]^T, one K16 step
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, Desc b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
        "mov.b64 db, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(leader)
        : "memory");
}
// Two K-major operands of 128 rows, D / 64 column halves 16 KB apart, 128-byte swizzle.
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t leader, uint32_t d, Desc a, Desc b, uint32_t idesc) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        const uint32_t at = (k / 4) * ((128 * 128) >> 4) + (k % 4) * 2;
        mma_ss(leader, d, Desc{a.lo + at, a.hi}, Desc{b.lo + at, b.hi}, idesc, k > 0 ? 1u : 0u);
    }
}
// Half h (64 of K) of A: 128 x 128 16-bit values in tensor memory, 32 columns for each half, A_STEP
// columns apart; B: 128 rows (K) in shared memory, MN-major.
template <int A_STEP>
__device__ __forceinline__ void mma_weights(uint32_t leader, uint32_t d, uint32_t a, Desc b, uint32_t idesc, uint32_t accumulate,
                                            int h) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
        mma_ts(leader, d, a + h * A_STEP + k * 8, Desc{b.lo + (4 * h + k) * (2048 >> 4), b.hi}, idesc, k > 0 ? 1u : accumulate);
}

// ------------------------------------------------------------------ e4m3
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
    return r;
}
__device__ __forceinline__ uint32_t floats_to_e4m3x2(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
    const uint32_t h = e4m3x2_to_half2(two);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// Two codes, times their scale, as bf16.  Exact for a power of two: a code has 4 significant
// bits, and bf16 has the exponents of fp32.  (Other scales round to nearest: taking the upper
// halves of the fp32 values, which is no faster, would cut them off.)
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two, float scale = 1.f) {
    const float2 f = e4m3x2_to_float2(two);
    return pack_bf16x2(f.x * scale, f.y * scale);
}
// 2^e for e in [-126, 127]
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

}  // namespace ac
