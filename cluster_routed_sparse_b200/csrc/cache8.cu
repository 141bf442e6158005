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

// Keys and values of the cache as bf16 rows [B, Hk, Lk, d], exact, for attention with
// many query rows: every 128-key tile that some query of the sequence sees, whole (zeros
// behind the sequence, where no query sees the page, and for bad pages).  A CTA takes one
// tile of one key head; bound by memory: 18,720 tokens of 12 heads, d = 128, 57 MB of codes
// to 115 MB of rows in 35 us, 4.9 TB/s.  Products of bf16 want no scales in the softmax.
template <int D>
__global__ void __launch_bounds__(kThreads) k_cache8_expand(const __grid_constant__ WinArgs a, bf16 *ko, bf16 *vo) {
    const int tiles = (a.Lk + 127) / 128;
    int idx = blockIdx.x;
    const int tile = idx % tiles;
    idx /= tiles;
    const int hk = idx % a.Hk, b = idx / a.Hk;
    const int ql = seq_len(a.q_lens, b, a.Lq, a.err), kl = seq_len(a.k_lens, b, a.Lk, a.err);
    if (ql == 0) return;
    const int lo = row_range(a.w, kl - ql, kl).lo, hi = row_range(a.w, kl - 1, kl).hi, sink = min(a.w.sinks, hi);
    const int base = tile * 128;
    if (base >= hi || (base + 128 <= lo && base >= sink)) return;
    const int log_t = 31 - __clz(a.T);
    // 8 codes at a time, so that a warp's stores fill whole sectors.
    constexpr int CPR = D / 8, N = 128 * CPR / kThreads;
    uint2 w[2][N];
    float sc[2][N];
#pragma unroll
    for (int c = 0; c < N; ++c) {
        const int ch = c * kThreads + threadIdx.x, key = base + ch / CPR, first = key >> log_t << log_t;
        w[0][c] = w[1][c] = make_uint2(0, 0);
        sc[0][c] = sc[1][c] = 0.f;
        if (key >= kl || !((first < hi && first + a.T > lo) || first < sink)) continue;
        const int page = __ldg(a.table + (int64_t)b * a.max_pages + (key >> log_t));
        if (page < 0 || page >= a.pages) {
            atomicOr(&a.err->bits, DEV_ERR_BOUNDS);
            continue;
        }
        const int64_t slot = (int64_t)page * a.Hk + hk, at = (slot * a.T + (key & (a.T - 1))) * D;
        w[0][c] = __ldg(reinterpret_cast<const uint2 *>(a.k8 + at) + ch % CPR);
        w[1][c] = __ldg(reinterpret_cast<const uint2 *>(a.v8 + at) + ch % CPR);
        sc[0][c] = __ldg(a.ks + slot), sc[1][c] = __ldg(a.vs + slot);
    }
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const int ch = c * kThreads + threadIdx.x, key = base + ch / CPR;
            if (key >= a.Lk) continue;
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t u = i < 2 ? w[v][c].x : w[v][c].y;
                r[i] = e4m3x2_to_bf16x2((u >> (16 * (i & 1))) & 0xFFFFu, sc[v][c]);
            }
            reinterpret_cast<uint4 *>((v ? vo : ko) + (((int64_t)b * a.Hk + hk) * a.Lk + key) * D)[ch % CPR] = make_uint4(r[0], r[1], r[2], r[3]);
        }
}

}  // namespace

cudaError_t launch_cache8_expand(const WinArgs &a, bf16 *k, bf16 *v, cudaStream_t s) {
    const int64_t grid = (int64_t)a.B * a.Hk * ((a.Lk + 127) / 128);
    if (grid == 0) return cudaSuccess;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (a.d == 128) k_cache8_expand<128><<<(unsigned)grid, kThreads, 0, s>>>(a, k, v);
    else k_cache8_expand<64><<<(unsigned)grid, kThreads, 0, s>>>(a, k, v);
    AC_NOTE_LAUNCH();
    return cudaGetLastError();
}

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
