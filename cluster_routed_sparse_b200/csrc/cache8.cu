// cache8.cu -- a paged cache of keys and values in 8 bits (e4m3), one scale for
// each page and head, and the append that fills it.
//
// The scale is a power of two, 2^e with the least e such that every value of
// the page fits in 448 * 2^e: a code times its scale is then exact in bf16 (4
// significant bits), so the attention that reads the cache rounds nothing, and
// when later tokens of a part-filled page need a larger scale, the earlier
// codes move by a power of two, exact except where they become subnormal.
//
// Bound by memory: 2 bytes read and 1 written per element.  One CTA holds one
// (page, head, K or V) in registers: loads, page maximum, conversion, stores; a page is
// the unit because its scale needs all of it.  14,400 tokens of 40 heads, d = 128, pages
// of 128 tokens (0.44 GB): 81 us, 5.5 TB/s, 84% of a copy (the loads of a page wait for
// nothing, its stores for the maximum; 512 threads a page: no better).  One token of
// eight sequences, 8 heads: 2.8 us in a graph.
#include "stream_device.cuh"

namespace ac {
namespace {

constexpr int kThreads = 256;
constexpr int kMinExp = -120, kMaxExp = 119;  // 448 * 2^119 is the largest that fp32 and bf16 hold

// NC chunks of 8 elements per thread: NC * kThreads * 8 >= T * D.
template <int D, int NC>
__global__ void __launch_bounds__(kThreads, NC > 4 ? 3 : 6) k_cache8_append(const AppendArgs a, int touched) {
    uint32_t idx = blockIdx.x;  // (page of the sequence, K or V, head, sequence)
    const int blk_i = idx % (uint32_t)touched;
    idx /= (uint32_t)touched;
    const bool is_v = idx & 1;
    idx >>= 1;
    const int h = idx % (uint32_t)a.Hk, b = idx / (uint32_t)a.Hk;
    const int start = a.start[b];
    int n = a.n;
    if (a.counts) {
        n = min(max(a.counts[b], 0), a.n);
        if (n != a.counts[b] && threadIdx.x == 0) atomicOr(&a.err->bits, DEV_ERR_BOUNDS);
    }
    if (start < 0) {
        if (threadIdx.x == 0) atomicOr(&a.err->bits, DEV_ERR_BOUNDS);
        return;
    }
    const int log_t = 31 - __clz(a.T);
    const int64_t blk = (start >> log_t) + blk_i;
    const int64_t first64 = blk * a.T - start;  // token index of the page's slot 0
    if (first64 >= n || n == 0) return;
    const int first = (int)first64;
    const int page = blk < a.max_pages ? a.table[(int64_t)b * a.max_pages + blk] : -1;
    if (page < 0 || page >= a.pages) {
        if (threadIdx.x == 0) atomicOr(&a.err->bits, DEV_ERR_BOUNDS);
        return;
    }
    constexpr int CPR = D / 8;  // chunks of a row
    const int chunks = a.T * CPR;
    const View &src = is_v ? a.v : a.k;
    const bf16 *x = static_cast<const bf16 *>(src.p) + b * src.b + h * src.h;
    const int64_t slot = (int64_t)page * a.Hk + h;
    uint8_t *codes = (is_v ? a.v8 : a.k8) + slot * a.T * D;
    float *scale = (is_v ? a.vs : a.ks) + slot;

    uint4 w[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int ch = c * kThreads + threadIdx.x, tok = first + ch / CPR;
        w[c] = make_uint4(0, 0, 0, 0);
        if (ch < chunks && tok >= 0 && tok < n) w[c] = *reinterpret_cast<const uint4 *>(x + tok * src.l + (ch % CPR) * 8);
    }
    // largest |value|: bf16 bits without the sign are ordered like the values
    uint32_t top2 = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const uint32_t u[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top2 = __vmaxu2(top2, u[i] & 0x7FFF7FFFu);
    }
    uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
    if (top > 0x7F80u) {  // a NaN, which has no size: once more without it
        top = 0;
        for (int c = 0; c < NC; ++c) {
            const uint32_t u[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = u[i] & 0x7FFFu, hi = (u[i] >> 16) & 0x7FFFu;
                top = max(top, max(lo > 0x7F80u ? 0u : lo, hi > 0x7F80u ? 0u : hi));
            }
        }
    }
    __shared__ uint32_t s_top;
    __shared__ int s_old;
    if (threadIdx.x == 0) {
        s_top = 0;
        s_old = (__float_as_int(*scale) >> 23) - 127;
    }
    __syncthreads();
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((threadIdx.x & 31) == 0) atomicMax(&s_top, top);
    __syncthreads();
    top = s_top;
    // 448 = 1.75 * 2^8: e = E - 8, one more when the significand is above 1.75
    int e = (int)(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u);
    e = min(max(e, kMinExp), kMaxExp);
    const int e_old = min(max(s_old, kMinExp), kMaxExp);
    const bool part = first < 0;  // earlier tokens share the page
    if (part) e = max(e, e_old);
    const float up = exp2i(-e);
    const int shift = e_old - e;  // <= 0 where it is used
    const float down = shift < -126 ? 0.f : exp2i(min(shift, 0));
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int ch = c * kThreads + threadIdx.x, tok = first + ch / CPR;
        if (ch >= chunks) continue;
        uint2 *dst = reinterpret_cast<uint2 *>(codes + ch * 8);
        if (tok >= 0 && tok < n) {
            const uint32_t u[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x0, x1;
                f2_unpack(f2_mul(f2_pack(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u)), f2_pack(up, up)), x0, x1);
                q[i] = floats_to_e4m3x2(x0, x1);
            }
            *dst = make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
        } else if (tok < 0 && shift < 0) {
            const uint2 old = *dst;
            const uint32_t u[2] = {old.x, old.y};
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = e4m3x2_to_float2((u[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
                q[i] = floats_to_e4m3x2(f.x * down, f.y * down);
            }
            *dst = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
        }
    }
    if (threadIdx.x == 0 && (!part || e != s_old)) *scale = exp2i(e);
}

}  // namespace

cudaError_t launch_cache8_append(const AppendArgs &a, cudaStream_t s) {
    const int touched = (a.n + a.T - 1) / a.T + 1;
    const int64_t grid = (int64_t)a.B * a.Hk * 2 * touched;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    auto go = [&](auto kern) { kern<<<(unsigned)grid, kThreads, 0, s>>>(a, touched); };
    const int nc = (a.T * a.d / 8 + kThreads - 1) / kThreads;
    if (a.d == 128)
        nc <= 1 ? go(k_cache8_append<128, 1>) : nc <= 2 ? go(k_cache8_append<128, 2>) : nc <= 4 ? go(k_cache8_append<128, 4>) : go(k_cache8_append<128, 8>);
    else
        nc <= 1 ? go(k_cache8_append<64, 1>) : nc <= 2 ? go(k_cache8_append<64, 2>) : go(k_cache8_append<64, 4>);
    AC_NOTE_LAUNCH();
    return cudaGetLastError();
}

}  // namespace ac
