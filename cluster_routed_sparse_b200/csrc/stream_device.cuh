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

// 5-D tiled bulk tensor load (coordinates x innermost).  No cluster multicast.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void *tmap, int32_t x, int32_t y, int32_t z, int32_t w,
                                            int32_t v, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar)
        : "memory");
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
// Over the cache, values whose page has a scale below 2^-90 count as zeros: the
// softmax sums divide by the scale and would leave fp32's range.
constexpr float kMinLogScale = -90.f, kMinScale = 8.077935669463161e-28f;
// 2^e for e in [-126, 127]
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

}  // namespace ac
